// bst_block_rows.hpp -- the block-scaled product for a few rows of A (a token,
// or some) and weights stored N x K.
//
// With few rows the weights are all there is to read, once, and the time is
// how many bytes are in flight.  A workgroup takes 16 columns of C, so that
// even one token's product over 4096 columns has a workgroup for every CU,
// and its eight waves share out K: each reads whole 128-byte blocks of its 16
// weight rows straight into the operand registers of the 16x16x128
// instruction (no LDS, no barrier in the loop, UNROLL blocks in flight per
// wave), and the waves' sums meet in LDS at the end, in wave order.  One
// launch and no workspace, where a split over workgroups needs two and one.
#pragma once

#include "bst_block_gemm.hpp"

namespace bst {

typedef float f32x4v_t __attribute__((ext_vector_type(4)));

template <int FM, int FN, bool EXACT>
struct BlockRows {
  static constexpr int NW = 8, NT = 64 * NW, UNROLL = FM * FN == 4 ? 2 : 4;

  // 16 codes at p, of which `left` are inside K; the rest may be anything
  // (inside the row's pitch) and become zeros.
  static __device__ __forceinline__ u32x4_t codes16(const uint8_t* p, int left) {
    if (left <= 0) return u32x4_t{0u, 0u, 0u, 0u};
    u32x4_t v = *(const u32x4_t*)p;
    if (left < 16) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int n = left - 4 * d;
        v[d] = n >= 4 ? v[d] : n <= 0 ? 0u : v[d] & ((1u << (8 * n)) - 1u);
      }
    }
    return v;
  }
  static __device__ __forceinline__ i32x8_t codes32(const uint8_t* p, int left) {
    const u32x4_t x = codes16(p, left), y = codes16(p + 16, left - 16);
    return i32x8_t{(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                   (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  }
  static __device__ __forceinline__ float scale(const uint8_t* s, int64_t at, bool f32) {
    return f32 ? ((const float*)s)[at] : e8m0_value(s[at]);
  }

  static __device__ __forceinline__ f32x4v_t product(const i32x8_t& b, const i32x8_t& a) {
    f32x4v_t p = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (EXACT) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(b, s), widen_codes(a, s), p, 0, 0, 0);
    } else {
      p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, p, 0, 0, 0, 0, 0, 0);
    }
    return p;
  }

  __device__ __attribute__((always_inline)) static void run(const BlockGemmArgs& a) {
    __shared__ f32x4v_t sums[FM * FN][NW][64];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    const uint32_t r = lane & 15u, q = lane >> 4;  // operand row; K 32q .. 32q+31 of a block
    const uint32_t n0 = blockIdx.x * (16u * FN);
    const uint8_t* b[FN];
    bool live_n[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const uint32_t n = n0 + j * 16 + r;
      live_n[j] = n < a.N;
      b[j] = a.B + (int64_t)(live_n[j] ? n : 0) * a.ldb + 32 * q;
    }
    const int64_t sb = (int64_t)(n0 / kScaleBlock) * a.ldsb;  // one block: 32 divides 128
    const uint8_t* ap[FM];
    int64_t sap[FM];
    bool live_m[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const uint32_t m = i * 16 + r;
      live_m[i] = m < a.M;
      ap[i] = a.A + (int64_t)(live_m[i] ? m : 0) * a.lda + 32 * q;
      sap[i] = (int64_t)(live_m[i] ? m : 0) * a.ldsa;
    }
    f32x4v_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4v_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t k0 = wave * UNROLL; k0 < a.nk; k0 += NW * UNROLL) {
      i32x8_t bv[UNROLL][FN], av[UNROLL][FM];
      float f[UNROLL][FM];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const uint32_t kb = k0 + u;
        const int64_t at = (int64_t)kb * 128;
        const int left = kb < a.nk ? (int)(a.K - kb * 128u) - 32 * (int)q : 0;
#pragma unroll
        for (int j = 0; j < FN; ++j) bv[u][j] = codes32(b[j] + at, live_n[j] ? left : 0);
        const float fb = kb < a.nk ? scale(a.sb, sb + kb, a.sb_f32 != 0) : 0.0f;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          av[u][i] = codes32(ap[i] + at, live_m[i] ? left : 0);
          f[u][i] = kb < a.nk ? scale(a.sa, sap[i] + kb, a.sa_f32 != 0) * fb : 0.0f;
        }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const f32x4v_t p = product(bv[u][j], av[u][i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(f[u][i], p[e], acc[i][j][e]);
          }
    }
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) sums[i * FN + j][wave][lane] = acc[i][j];
    __syncthreads();
    // wave w ends fragment (w / FN, w % FN); lane l: row l & 15 of it, columns
    // 4 (l >> 4) + 0..3
    if (wave >= (uint32_t)(FM * FN)) return;
    f32x4v_t s = sums[wave][0][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += sums[wave][w][lane];
    const uint32_t m = wave / FN * 16 + r, c = n0 + wave % FN * 16 + 4 * q;
    if (m >= a.M || c >= a.N) return;
    const int64_t es = a.ckind == OUT_F32 ? 4 : 2;
    float v[4] = {s[0], s[1], s[2], s[3]};
    put_run<4>(a.C + ((int64_t)m * a.ldc + c) * es, nullptr, v, a.N - c,
               a.cvec != 0 && a.N - c >= 4u, a.ckind);
  }
};

template <int FM, int FN, bool EXACT>
__global__ void __launch_bounds__(512) block_rows_kernel(BlockGemmArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  BlockRows<FM, FN, EXACT>::run(a);
#endif
}

}  // namespace bst
