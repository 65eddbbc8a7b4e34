/*
 * bst_block.h -- C ABI of the block-scaled 8-bit operators: matrices of OCP
 * FP8 E4M3 codes with one scale for each block of 128, as 8-bit checkpoints
 * of language models are published and trained, and what a linear layer
 * computes with them forward and backward.
 *
 * An 8-bit matrix is a row-major code matrix Q and a scale matrix S:
 *   activations  S [M][ceil(K/128)]            one scale per row and 128 columns
 *   weights      S [ceil(K/128)][ceil(N/128)]  one scale per 128 x 128 square
 * and stands for Q[i][j] times the scale of its block.  The last block of a
 * row or column may be shorter.  A scale is either
 *   BST_E8M0  one byte e for 2^(e - 127) (255: NaN), or
 *   BST_F32   a 32-bit float of any value.
 *
 * The conventions of bst.h hold: the caller owns every buffer and the
 * stream, nothing is allocated or synchronised in a call, all arguments are
 * checked before anything is enqueued, bst_last_error() describes a failure.
 * Further:
 *  - Code matrices (A, B, Q of the products and gradients) need 16-byte
 *    aligned bases and leading dimensions that are multiples of 16; any
 *    M, N, K.  Bytes between a row's end and its pitch are never used, so
 *    they may hold anything.  Other matrices (X, dY, C, dW, add) may have
 *    any element-aligned base and any pitch >= the row length; 16-byte
 *    aligned rows are faster.
 *  - Outputs may not overlap inputs, except where a call says so.  Calls run on
 *    the device that is current; operands, workspace and stream belong to it.
 *  - Sums are held in fp32 and rounded once to the output type, to nearest
 *    even; what the 8-bit matrix instruction drops on the way is stated at
 *    bst_gemm_block_scaled.  Results do not depend on the schedule except for the order of
 *    the fp32 sums, and two calls with the same arguments give the same bits.
 *  - A workspace needs no initialisation: nothing that it holds before a call
 *    enters a result (only the columns that pad its rows are read unwritten,
 *    and thrown away).  It is in use until the
 *    call's work on the stream is done: calls that may run at the same time
 *    need a workspace each.
 *  - Every call may be captured into a graph: it only launches kernels.
 *  - BST_E_UNSUPPORTED where a call would need more threads than a launch
 *    holds (2^32; e.g. more than 2^23 output tiles), BST_E_INVAL where a split
 *    output has more than 2^33 values, or a matrix to quantise or restore more
 *    than 2^31 - 1 runs of 128 in its rows.
 */
#ifndef BST_BLOCK_H
#define BST_BLOCK_H

#include "bst.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BST_E8M0 ((bst_dtype)8) /* scale type: 2^(byte - 127) */

/*
 * bst_quant_block -- 8-bit codes and scales of X [M][ldx].
 *   x: BST_BF16, BST_F16 or BST_F32.  block_rows: 1 (blocks of 128
 *   consecutive values of a row) or 128 (128 x 128 squares).
 *   Q [M][ldq] e4m3 codes; S [ceil(M/block_rows)][lds] E8M0 bytes.
 *   A block's scale is 2^e with the smallest e >= -127 such that its largest
 *   finite magnitude is at most 448 * 2^e; a code is x * 2^-e rounded to
 *   nearest even.  Powers of two make this exact apart from that one
 *   rounding, and make the restored values exact in bf16.  Infinities and
 *   NaN become the code NaN and do not enter the scale.
 *   Q and S may not overlap X.
 */
bst_status bst_quant_block(bst_dtype x, int64_t M, int64_t K, int32_t block_rows,
                           const void* X_dev, int64_t ldx, uint8_t* Q_dev, int64_t ldq,
                           uint8_t* S_dev, int64_t lds, void* stream);

/*
 * bst_dequant_block -- X = Q times its blocks' scales, rounded to x
 * (BST_BF16, BST_F16 or BST_F32); s: BST_E8M0 or BST_F32.  A code times a
 * 32-bit scale is rounded to fp32 before it is rounded to x.  A finite code
 * times a finite scale that leaves x's range gives x's largest finite value
 * with its sign (65504 * 2^-8 may round up in 8 bits), never an infinity.
 */
bst_status bst_dequant_block(bst_dtype x, int64_t M, int64_t K, int32_t block_rows,
                             const uint8_t* Q_dev, int64_t ldq, bst_dtype s, const void* S_dev,
                             int64_t lds, void* X_dev, int64_t ldx, void* stream);

/*
 * bst_gemm_block_scaled -- C [M][N] = A . B of two 8-bit matrices:
 *   C[i][j] = sum over K blocks b of sa[i][b] * sb[b][j/128] *
 *             (sum over the block's k of A[i][k] * B[k][j]).
 *   A [M][lda] codes, SA [M][ldsa] scales of type sa (one per row and block).
 *   trans_b = 0: B [K][ldb], SB [ceil(K/128)][ldsb];
 *   trans_b = 1: B [N][ldb] (the transposed matrix), SB [ceil(N/128)][ldsb].
 *   The same weight in one storage order serves the forward product and, with
 *   the other value of trans_b, the gradient of the input (dX = dY . W^T).
 *   sa and sb are BST_E8M0 or BST_F32 each.  The product of the two scales of
 *   a sum must lie in the range of fp32.
 *   c: BST_BF16, BST_F16 or BST_F32.  The 8-bit matrix instructions behind
 *   bf16 and fp16 outputs add 8 consecutive products at the largest one's
 *   exponent and drop what is below 2^-13 of that (about 1.5e-5 of a result,
 *   and more of one whose terms cancel); an fp32 output is computed on bf16
 *   instructions from the same codes, which keep fp32 throughout, and takes
 *   about twice as long, on large products three times (8192 x 8192 x 4096,
 *   E8M0: 229 us with bf16 out, 725 with fp32).
 *   A few rows of A (at most 32, or 64 with trans_b = 0) run on kernels of
 *   their own where K and N are not too long and no tile or split is asked for; they
 *   read every weight once, in one launch and without a workspace.
 *   sched: NULL, or a schedule of which tile_m x tile_n (0 x 0 = chosen by
 *   the sizes; 32x128, 64x128, 128x128, and 256x256 for 16-bit outputs), swizzle_offset,
 *   swizzle_direction, xcd_remap and split_k (0 = chosen, at most 64) are used; tile_k
 *   is 0 or 128 and grid, path, shuffle_k, dynamic and preload are 0
 *   (BST_E_UNSUPPORTED otherwise).
 *   ws: bst_block_workspace_bytes(0, or 3 with trans_b = 1, ...) bytes,
 *   16-byte aligned (may be NULL when that is 0).
 *   BST_E_UNSUPPORTED if 256 rows of A or B (with trans_b = 0: 128 rows of
 *   B) span 2 GiB.
 */
bst_status bst_gemm_block_scaled(bst_dtype c, int32_t trans_b, int64_t M, int64_t N, int64_t K,
                                 const uint8_t* A_dev, int64_t lda, bst_dtype sa,
                                 const void* SA_dev, int64_t ldsa, const uint8_t* B_dev,
                                 int64_t ldb, bst_dtype sb, const void* SB_dev, int64_t ldsb,
                                 void* C_dev, int64_t ldc, const bst_sched* sched, void* ws,
                                 size_t ws_bytes, void* stream);

/*
 * bst_grouped_gemm_block_scaled -- the same (with the same instructions for
 * each output type) for G groups of rows stacked
 * along M, as bst_grouped_gemm_slice_m: rows [P_g, P_g + group_m[g]) of A and
 * C belong to group g and are multiplied by B_g = B + g*strideB (bytes) with
 * scales SB + g*strideSB (elements).  group_m_dev: device int32 [G], never
 * read by the host; entries < 0 count as 0 and groups are cut to total_m
 * rows.  Rows of C past the last group are left as they were.
 * 1 <= G <= 1024; sched->split_k must be 0 or 1.  Needs no workspace.
 */
bst_status bst_grouped_gemm_block_scaled(bst_dtype c, int32_t trans_b, int32_t G,
                                         const int32_t* group_m_dev, int64_t total_m, int64_t N,
                                         int64_t K, const uint8_t* A_dev, int64_t lda,
                                         bst_dtype sa, const void* SA_dev, int64_t ldsa,
                                         const uint8_t* B_dev, int64_t ldb, int64_t strideB,
                                         bst_dtype sb, const void* SB_dev, int64_t ldsb,
                                         int64_t strideSB, void* C_dev, int64_t ldc,
                                         const bst_sched* sched, void* stream);

/*
 * bst_weight_grad -- dW [K][N] = add + X^T . dY, the gradient of a linear
 * layer's weight from its input kept in 8 bits: X [M][K] is the matrix that
 * bst_quant_block with block_rows = 1 made (codes Q [M][ldq], E8M0 scales
 * S [M][lds]), dY [M][lddy] is the output's gradient in bf16, fp16 or fp32.
 *   dW[k][n] = add[k][n] + sum over m of X[m][k] * dY[m][n].
 *   X is what bst_dequant_block gives in bf16: exact above 2^-133, and where a
 *   code times its scale is past bf16's range, bf16's largest value.  The
 *   products run on bf16 matrix instructions: a bf16 dY as it is, an fp16 or
 *   fp32 dY as two or three bf16 parts that add up to it (exactly, down to
 *   2^-133), so no operand is rounded.
 *   dw: BST_F32, BST_BF16 or BST_F16.  add_dev: NULL, or a matrix of dW's
 *   type and layout ([K][ldadd]); it may be dW itself.  M = 0 gives add (or 0).
 *   tile_m x tile_n of sched: 128x128 or 256x256 (tile_m along K, tile_k 0);
 *   the other fields as for bst_gemm_block_scaled, split_k along M.
 *   ws: bst_block_workspace_bytes(1, ...) bytes.
 *   BST_E_UNSUPPORTED if 64 rows of Q span 2 GiB.
 */
bst_status bst_weight_grad(bst_dtype dy, bst_dtype dw, int64_t M, int64_t N, int64_t K,
                           const uint8_t* Q_dev, int64_t ldq, const uint8_t* S_dev, int64_t lds,
                           const void* dY_dev, int64_t lddy, const void* add_dev, int64_t ldadd,
                           void* dW_dev, int64_t lddw, const bst_sched* sched, void* ws,
                           size_t ws_bytes, void* stream);

/*
 * bst_grouped_weight_grad -- one gradient per group of rows: dW_g = add_g +
 * X_g^T . dY_g over rows [P_g, P_g + group_m[g]) (as in
 * bst_grouped_gemm_block_scaled; groups of any size; where a few groups hold
 * most rows, a schedule with xcd_remap = 0 is faster).  dW_g = dW +
 * g*stridedw, add_g = add + g*strideadd (elements).  An empty group's
 * gradient is add_g (or 0).  ws: bst_block_workspace_bytes(2, ...) bytes.
 */
bst_status bst_grouped_weight_grad(bst_dtype dy, bst_dtype dw, int32_t G,
                                   const int32_t* group_m_dev, int64_t total_m, int64_t N,
                                   int64_t K, const uint8_t* Q_dev, int64_t ldq,
                                   const uint8_t* S_dev, int64_t lds, const void* dY_dev,
                                   int64_t lddy, const void* add_dev, int64_t ldadd,
                                   int64_t strideadd, void* dW_dev, int64_t lddw,
                                   int64_t stridedw, const bst_sched* sched, void* ws,
                                   size_t ws_bytes, void* stream);

/*
 * bst_block_workspace_bytes -- workspace bytes of a call with these sizes on
 * the current device: kind 0 bst_gemm_block_scaled with trans_b = 0, 3 with
 * trans_b = 1, 1 bst_weight_grad, 2 bst_grouped_weight_grad (count = G, M =
 * total_m).  0 where no split runs, and for invalid arguments (with the last
 * error set).
 */
size_t bst_block_workspace_bytes(int kind, int64_t count, int64_t M, int64_t N, int64_t K,
                                 const bst_sched* sched);

#ifdef __cplusplus
}
#endif

#endif /* BST_BLOCK_H */
