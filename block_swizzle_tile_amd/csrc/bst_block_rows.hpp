// bst_block_rows.hpp -- the block-scaled product for a few rows of A (a token,
// or some): BlockRows for weights stored N x K, BlockRowsN for K x N.
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

// ------------------------------------------------------- weights K x N ----
// The same for weights whose rows run along N: an operand then has to be
// gathered from 128 rows, which the transposing LDS reads do.  A workgroup
// takes 32 columns; its eight waves share out the blocks of K, and each runs
// a pipeline of its own (DMA of the wave's next 128 x 32 patch into its own
// two LDS buffers while it multiplies the last one), so that the loop has no
// barrier and eight patches are in flight per workgroup.  The 32-byte rows of
// a patch share their cache lines with the neighbours', which run on the same
// die.  64 columns were slower (33 rows, 4112 x 2056: 8.4 us against 7.0), and
// so were 16 waves (9.8).  A comes straight from memory: a lane's 32 bytes of
// each half block.
template <int FM, bool EXACT>
struct BlockRowsN {
  static constexpr int NW = 8, BN = 32;
  static constexpr int BUF = 128 * BN;  // a patch
  static constexpr int SUMS = FM * 32 * BN * 4;  // a wave's partial sums
  static constexpr int LDS_BYTES = NW * (2 * BUF > SUMS ? 2 * BUF : SUMS);
  static_assert(LDS_BYTES <= 160 * 1024, "LDS budget");
  using Rows = BlockRows<1, 1, EXACT>;

  static __device__ __forceinline__ lds_t* lds() {
    __shared__ __attribute__((aligned(16))) uint8_t buf[LDS_BYTES];
    return (lds_t*)buf;
  }
  // XOR of a row's chunks: rows 0..7 of a transposing read fall on all banks
  static constexpr int CPR = BN / 16, RPI = 64 / CPR, DMAS = 128 / RPI;
  static __device__ __forceinline__ uint32_t swz_n(uint32_t k) { return (k >> 2) & 1u; }

  struct Next {
    i32x8_t a[2][FM];
    float f[FM];
  };

  __device__ __attribute__((always_inline)) static void run(const BlockGemmArgs& a) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t l32 = lane & 31u, hi = lane >> 5;
    const uint32_t n0 = logical_wg(1u, a.grid) * BN;
    const uint32_t cols = a.N - n0 < (uint32_t)BN ? a.N - n0 : BN;
    const int64_t sb = n0 / kScaleBlock;  // one block of columns: 32 divides 128
    lds_t* const own = lds() + wave * (2 * BUF);
    // DMA instruction x: K rows RPI x + lane / CPR, chunk lane % CPR of the patch
    const uint32_t dk = lane / CPR, dch = (lane % CPR) ^ swz_n(dk);
    const uint32_t doff = dch * 16 < cols ? dk * (uint32_t)a.ldb + dch * 16 : kOob;
    // transposing reads: K = 64 kk + 32 (t >> 1) + 16 hi + 8 (t & 1) + (L >> 1)
    const uint32_t L = lane & 15u, rk = 16 * hi + (L >> 1);
    const uint32_t roff = rk * BN + ((((lane >> 4) & 1u) ^ swz_n(rk)) << 4) + 8 * (L & 1u);

    auto fetch = [&](uint32_t kb, uint32_t s, Next& n) {
      const uint32_t left = a.K - kb * 128u;  // > 0
      const u32x4_t d = make_desc(a.B + (int64_t)kb * 128 * a.ldb + n0);
#pragma unroll
      for (int x = 0; x < DMAS; ++x)
        dma16(d, own + s * BUF + x * 1024, RPI * x + dk < left ? doff : kOob,
              (uint32_t)(RPI * x) * (uint32_t)a.ldb);
      const float fb = Rows::scale(a.sb, sb + (int64_t)kb * a.ldsb, a.sb_f32 != 0);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const uint32_t m = i * 32 + l32;
        const bool live = m < a.M;
        const int64_t row = live ? m : 0;
        n.f[i] = Rows::scale(a.sa, row * a.ldsa + kb, a.sa_f32 != 0) * fb;
        const uint8_t* p = a.A + row * a.lda + (int64_t)kb * 128;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const int k = 64 * kk + 16 * (int)hi;
          const u32x4_t x = Rows::codes16(p + k, live ? (int)left - k : 0);
          const u32x4_t y = Rows::codes16(p + k + 32, live ? (int)left - k - 32 : 0);
          n.a[kk][i] = i32x8_t{(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                               (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
        }
      }
    };

    f32x16_t acc[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
    Next next;
    uint32_t s = 0;
    if (wave < a.nk) fetch(wave, 0, next);
    for (uint32_t kb = wave; kb < a.nk; kb += NW) {
      const Next now = next;
      // this patch has landed, and the other buffer's reads are done
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      if (kb + NW < a.nk) fetch(kb + NW, s ^ 1u, next);
      i32x8_t b[2];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        i32x2_t v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          v[t] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (lds_i32x2_t*)(own + s * BUF + roff + (64 * kk + 32 * (t >> 1) + 8 * (t & 1)) * BN));
        b[kk] = i32x8_t{v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]};
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        f32x16_t p = {};
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          if constexpr (EXACT) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_codes(b[kk], u),
                                                          widen_codes(now.a[kk][i], u), p, 0, 0, 0);
          } else {
            p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[kk], now.a[kk][i], p, 0, 0, 0, 0,
                                                                0, 0);
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] = __builtin_fmaf(now.f[i], p[e], acc[i][e]);
      }
      s ^= 1u;
    }
    // ---- the waves' sums, each in rows of BN columns whose 4-column chunks
    // are XORed by the row, then added in wave order
    constexpr uint32_t QPR = BN / 4;
    __syncthreads();
    typedef __attribute__((address_space(3))) f32x4_t lds_f4_t;
    lds_t* const mine = lds() + wave * SUMS;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t m = i * 32 + l32, ch = 2 * q + hi;
        *(lds_f4_t*)(mine + m * (BN * 4) + ((ch ^ (m & (QPR - 1))) << 4)) =
            f32x4_t{acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]};
      }
    __syncthreads();
    const int64_t es = a.ckind == OUT_F32 ? 4 : 2;
    for (uint32_t id = threadIdx.x; id < FM * 32 * QPR; id += NW * 64) {
      const uint32_t m = id / QPR, ch = id % QPR, c = ch * 4;
      if (m >= a.M || c >= cols) continue;
      const lds_t* p = lds() + m * (BN * 4) + ((ch ^ (m & (QPR - 1))) << 4);
      f32x4_t t = *(const lds_f4_t*)p;
#pragma unroll
      for (int w = 1; w < NW; ++w) t += *(const lds_f4_t*)(p + w * SUMS);
      float v[4] = {t[0], t[1], t[2], t[3]};
      put_run<4>(a.C + ((int64_t)m * a.ldc + n0 + c) * es, nullptr, v, cols - c,
                 a.cvec != 0 && cols - c >= 4u, a.ckind);
    }
  }
};

template <int FM, bool EXACT>
__global__ void __launch_bounds__(512) block_rows_n_kernel(BlockGemmArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  BlockRowsN<FM, EXACT>::run(a);
#endif
}

}  // namespace bst
