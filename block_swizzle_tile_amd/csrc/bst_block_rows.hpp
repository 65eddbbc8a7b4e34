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

template <int FM, bool EXACT>
struct BlockRows {
  static constexpr int NW = 8, UNROLL = 4;

  // Loads have no branches around them, so that all of a step's are in flight
  // together: a lane without data gives an offset out of the buffer's range and
  // gets zeros.
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), (short)0, (int)kOob, 0x00020000);
  }
  // 16 codes, if any of them is inside K (left > 0)
  static __device__ __forceinline__ u32x4_t codes16(__amdgpu_buffer_rsrc_t r, uint32_t at,
                                                    uint32_t uniform_at, int left) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, left > 0 ? at : kOob, uniform_at, 0);
  }
  // `left` of 16 codes are inside K; the rest may be anything (inside the row's
  // pitch) and become zeros.
  static __device__ __forceinline__ void cut(int* v, int left) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int n = left - 4 * d;
      v[d] = n >= 4 ? v[d] : n <= 0 ? 0 : (int)((uint32_t)v[d] & ((1u << (8 * n)) - 1u));
    }
  }
  static __device__ __forceinline__ void cut32(i32x8_t& v, int left) {
    int w[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    cut(w, left);
    cut(w + 4, left - 16);
    v = i32x8_t{w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
  }
  static __device__ __forceinline__ i32x8_t codes32(__amdgpu_buffer_rsrc_t r, uint32_t at,
                                                    uint32_t uniform_at, int left) {
    const u32x4_t x = codes16(r, at, uniform_at, left);
    const u32x4_t y = codes16(r, at + 16, uniform_at, left - 16);
    return i32x8_t{(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                   (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  }
  // A scale's bits (at: elements), and its value.
  static __device__ __forceinline__ uint32_t scale_bits(__amdgpu_buffer_rsrc_t r, uint32_t at, bool f32) {
    if (f32) return __builtin_amdgcn_raw_buffer_load_b32(r, at * 4u, 0, 0);
    return __builtin_amdgcn_raw_buffer_load_b8(r, at, 0, 0);
  }
  static __device__ __forceinline__ float scale_value(uint32_t bits, bool f32) {
    return f32 ? __builtin_bit_cast(float, bits) : e8m0_value(bits);
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
    __shared__ f32x4v_t sums[FM][NW][64];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    const uint32_t r = lane & 15u, q = lane >> 4;  // operand row; K 32q .. 32q+31 of a block
    const uint32_t n0 = blockIdx.x * 16u;
    // rows past N or M read row 0's scales; their codes are zeros
    const bool live_n = n0 + r < a.N;
    const uint32_t bo = r * (uint32_t)a.ldb + 32 * q;
    uint32_t ao[FM], so[FM];
    bool live_m[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const uint32_t m = i * 16 + r;
      live_m[i] = m < a.M;
      ao[i] = m * (uint32_t)a.lda + 32 * q;
      so[i] = live_m[i] ? m * (uint32_t)a.ldsa : 0u;
    }
    const __amdgpu_buffer_rsrc_t rb = buffer(a.B + (int64_t)n0 * a.ldb), ra = buffer(a.A), rsa = buffer(a.sa);
    // one block of columns: 16 divides 128
    const __amdgpu_buffer_rsrc_t rsb =
        buffer(a.sb + (int64_t)(n0 / kScaleBlock) * a.ldsb * (a.sb_f32 ? 4 : 1));
    const bool sa_f32 = a.sa_f32 != 0, sb_f32 = a.sb_f32 != 0;
    f32x4v_t acc[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) acc[i] = f32x4v_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t k0 = wave * UNROLL; k0 < a.nk; k0 += NW * UNROLL) {
      i32x8_t bv[UNROLL], av[UNROLL][FM];
      uint32_t sav[UNROLL][FM], sbv[UNROLL];
      auto left = [&](int u) {
        return k0 + u < a.nk ? (int)(a.K - (k0 + u) * 128u) - 32 * (int)q : 0;
      };
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const uint32_t at = (k0 + u) * 128u;
        bv[u] = codes32(rb, bo, at, live_n ? left(u) : 0);
#pragma unroll
        for (int i = 0; i < FM; ++i) av[u][i] = codes32(ra, ao[i], at, live_m[i] ? left(u) : 0);
      }
      // blocks past the last read its scales again; their codes are zeros
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) sbv[u] = scale_bits(rsb, min(k0 + u, a.nk - 1), sb_f32);
#pragma unroll
      for (int u = 0; u < UNROLL; ++u)
#pragma unroll
        for (int i = 0; i < FM; ++i) sav[u][i] = scale_bits(rsa, so[i] + min(k0 + u, a.nk - 1), sa_f32);
      if ((a.K & 15u) != 0 && k0 + UNROLL >= a.nk) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          if (k0 + u + 1 != a.nk) continue;
          cut32(bv[u], left(u));
#pragma unroll
          for (int i = 0; i < FM; ++i) cut32(av[u][i], left(u));
        }
      }
      float f[UNROLL][FM];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const float fb = k0 + u < a.nk ? scale_value(sbv[u], sb_f32) : 0.0f;
#pragma unroll
        for (int i = 0; i < FM; ++i)
          f[u][i] = k0 + u < a.nk ? scale_value(sav[u][i], sa_f32) * fb : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u)
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const f32x4v_t p = product(bv[u], av[u][i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(f[u][i], p[e], acc[i][e]);
        }
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) sums[i][wave][lane] = acc[i];
    __syncthreads();
    // wave w ends fragment w; lane l: row l & 15 of it, columns 4 (l >> 4) + 0..3
    if (wave >= (uint32_t)FM) return;
    f32x4v_t s = sums[wave][0][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += sums[wave][w][lane];
    const uint32_t m = wave * 16 + r, c = n0 + 4 * q;
    if (m >= a.M || c >= a.N) return;
    const int64_t es = a.ckind == OUT_F32 ? 4 : 2;
    float v[4] = {s[0], s[1], s[2], s[3]};
    put_run<4>(a.C + ((int64_t)m * a.ldc + c) * es, nullptr, v, a.N - c,
               a.cvec != 0 && a.N - c >= 4u, a.ckind);
  }
};

template <int FM, bool EXACT>
__global__ void __launch_bounds__(512) block_rows_kernel(BlockGemmArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  BlockRows<FM, EXACT>::run(a);
#endif
}

// ------------------------------------------------------- weights K x N ----
// The same for weights whose rows run along N: an operand then has to be
// gathered from 128 rows, which the transposing LDS reads do.  A workgroup
// takes 32 columns; its eight waves share out the blocks of K, and each asks
// for all of its 128 x 32 patches (up to four, by DMA into its own LDS buffers)
// before it multiplies the first, so that the time is about one memory latency
// (33 rows, 4112 x 2056: 7.8 us with two buffers a wave, 6.4 with four) and
// there is no barrier before the sums.  The 32-byte rows of a patch share their
// cache lines with the neighbours', which run on the same die.  With two
// buffers, 64 columns a workgroup were slower (8.4 us against 7.0), and so were
// 16 waves (9.8).  A comes straight from memory: a lane's 32 bytes of each half
// block.
template <int FM, bool EXACT>
struct BlockRowsN {
  static constexpr int NW = 8, BN = 32, DEPTH = 4;
  static constexpr int MOST = NW * DEPTH;  // blocks of K: a buffer for every patch
  static constexpr int BUF = 128 * BN;  // a patch
  static constexpr int SUMS = FM * 32 * BN * 4;  // a wave's partial sums
  static constexpr int LDS_BYTES = NW * (DEPTH * BUF > SUMS ? DEPTH * BUF : SUMS);
  static_assert(LDS_BYTES <= 160 * 1024, "LDS budget");
  using Rows = BlockRows<1, EXACT>;

  static __device__ __forceinline__ lds_t* lds() {
    __shared__ __attribute__((aligned(16))) uint8_t buf[LDS_BYTES];
    return (lds_t*)buf;
  }
  // XOR of a row's chunks: rows 0..7 of a transposing read fall on all banks
  static constexpr int CPR = BN / 16, RPI = 64 / CPR, DMAS = 128 / RPI;
  static __host__ __device__ __forceinline__ uint32_t swz_n(uint32_t k) { return (k >> 2) & 1u; }

  // A lane's part of the addressing (it runs on the host too, where a test checks
  // every access).  DMA instruction x: K rows RPI x + lane / CPR, chunk lane % CPR
  // of the patch.
  struct Lane {
    uint32_t k, off;  // first K row, and its offset from the patch's (kOob: past the columns)
  };
  static __host__ __device__ __forceinline__ Lane dma_lane(uint32_t lane, uint32_t ldb32, uint32_t cols) {
    const uint32_t k = lane / CPR, ch = (lane % CPR) ^ swz_n(k);
    return Lane{k, ch * 16 < cols ? k * ldb32 + ch * 16 : kOob};
  }
  // left: K rows from the patch's first on
  static __host__ __device__ __forceinline__ uint32_t dma_voff(const Lane& l, int x, uint32_t left) {
    return RPI * x + l.k < left ? l.off : kOob;
  }
  static __host__ __device__ __forceinline__ uint32_t dma_soff(int x, uint32_t ldb32) {
    return (uint32_t)(RPI * x) * ldb32;
  }
  // transposing reads: K = 64 kk + 32 (t >> 1) + 16 hi + 8 (t & 1) + (L >> 1)
  static __host__ __device__ __forceinline__ uint32_t read_off(uint32_t lane) {
    const uint32_t L = lane & 15u, rk = 16 * (lane >> 5) + (L >> 1);
    return rk * BN + ((((lane >> 4) & 1u) ^ swz_n(rk)) << 4) + 8 * (L & 1u);
  }
  static __host__ __device__ constexpr uint32_t read_step(int kk, int t) {
    return (64 * kk + 32 * (t >> 1) + 8 * (t & 1)) * BN;
  }

  // A's part of a patch.
  struct Rest {
    i32x8_t a[2][FM];
    uint32_t sa[FM], sb;
  };
  // At least these many accesses of a patch are in the wave's queue (its scales
  // come on top).
  static constexpr int QUEUED = DMAS + 4 * FM;
  static_assert((DEPTH - 1) * QUEUED < 64, "vmcnt holds 6 bits");
  // The oldest patch has landed, with LATER others behind it.
  template <int LATER>
  static __device__ __forceinline__ void wait_for() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LATER * QUEUED) : "memory");
  }

  __device__ __attribute__((always_inline)) static void run(const BlockGemmArgs& a) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t l32 = lane & 31u, hi = lane >> 5;
    const uint32_t n0 = logical_wg(1u, a.grid) * BN;
    const uint32_t cols = a.N - n0 < (uint32_t)BN ? a.N - n0 : BN;
    const int64_t sb = n0 / kScaleBlock;  // one block of columns: 32 divides 128
    lds_t* const own = lds() + wave * (DEPTH * BUF);
    const Lane dl = dma_lane(lane, (uint32_t)a.ldb, cols);
    const uint32_t roff = read_off(lane);
    const bool sa_f32 = a.sa_f32 != 0, sb_f32 = a.sb_f32 != 0;
    const __amdgpu_buffer_rsrc_t ra = Rows::buffer(a.A), rsa = Rows::buffer(a.sa);
    uint32_t ao[FM], so[FM];
    bool live[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const uint32_t m = i * 32 + l32;
      live[i] = m < a.M;
      ao[i] = m * (uint32_t)a.lda + 16 * hi;
      so[i] = live[i] ? m * (uint32_t)a.ldsa : 0u;
    }

    auto fetch = [&](uint32_t kb, uint32_t s, Rest& n) {
      const uint32_t left = a.K - kb * 128u;  // > 0
      const u32x4_t d = make_desc(a.B + (int64_t)kb * 128 * a.ldb + n0);
#pragma unroll
      for (int x = 0; x < DMAS; ++x)
        dma16(d, own + s * BUF + x * 1024, dma_voff(dl, x, left), dma_soff(x, (uint32_t)a.ldb));
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const int have = live[i] ? (int)left - 64 * kk - 16 * (int)hi : 0;
          const u32x4_t x = Rows::codes16(ra, ao[i] + 64 * kk, kb * 128u, have);
          const u32x4_t y = Rows::codes16(ra, ao[i] + 64 * kk + 32, kb * 128u, have - 32);
          n.a[kk][i] = i32x8_t{(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                               (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
        }
      n.sb = Rows::scale_bits(Rows::buffer(a.sb + (sb + (int64_t)kb * a.ldsb) * (sb_f32 ? 4 : 1)), 0, sb_f32);
#pragma unroll
      for (int i = 0; i < FM; ++i) n.sa[i] = Rows::scale_bits(rsa, so[i] + kb, sa_f32);
    };

    f32x16_t acc[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
    auto multiply = [&](uint32_t kb, uint32_t s, Rest& n) {
      if (a.K - kb * 128u < 128u && (a.K & 15u) != 0) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const int have = (int)(a.K - kb * 128u) - 64 * kk - 16 * (int)hi;
            int w[8];
#pragma unroll
            for (int d = 0; d < 8; ++d) w[d] = n.a[kk][i][d];
            Rows::cut(w, have);
            Rows::cut(w + 4, have - 32);
            n.a[kk][i] = i32x8_t{w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
          }
      }
      i32x8_t b[2];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        i32x2_t v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          v[t] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (lds_i32x2_t*)(own + s * BUF + roff + read_step(kk, t)));
        b[kk] = i32x8_t{v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]};
      }
      const float fb = Rows::scale_value(n.sb, sb_f32);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        f32x16_t p = {};
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          if constexpr (EXACT) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_codes(b[kk], u),
                                                          widen_codes(n.a[kk][i], u), p, 0, 0, 0);
          } else {
            p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[kk], n.a[kk][i], p, 0, 0, 0, 0, 0, 0);
          }
        }
        const float f = Rows::scale_value(n.sa[i], sa_f32) * fb;
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] = __builtin_fmaf(f, p[e], acc[i][e]);
      }
    };

    // patch t of the wave is block wave + t NW of K, in buffer t
    const uint32_t count = wave < a.nk ? (a.nk - wave + NW - 1) / NW : 0u;
    Rest rest[DEPTH];
    static_for<DEPTH>([&](auto u) {
      constexpr uint32_t U = decltype(u)::value;
      if (U < count) fetch(wave + U * NW, U, rest[U]);
    });
    static_for<DEPTH>([&](auto u) {
      constexpr uint32_t U = decltype(u)::value;
      if (U >= count) return;
      const uint32_t later = count - 1 - U;
      if (later >= 3) wait_for<3>();
      else if (later == 2) wait_for<2>();
      else if (later == 1) wait_for<1>();
      else wait_for<0>();
      multiply(wave + U * NW, U, rest[U]);
    });
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
