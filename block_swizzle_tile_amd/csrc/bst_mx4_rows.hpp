// bst_mx4_rows.hpp -- the 4-bit product for a few rows of A (a token, or some).
//
// With few rows the weights are all there is to read, once, and the time is how
// many bytes are in flight.  A workgroup takes 16 columns of C, so that even one
// token's product over 4096 columns has a workgroup for every CU, and its eight
// waves share out K: each reads whole 128-byte lines of its 16 weight rows
// straight into the operand registers of the 16x16x128 instruction (no LDS, no
// barrier in the loop), and the waves' sums meet in LDS at the end, in wave
// order.  One launch and no workspace, where a split over workgroups needs two
// and one.
//
// Grouped (a mixture of experts that serves a few tokens), a workgroup takes 16
// columns of one group's weights and 16 FM of its rows.  Every group has workgroups
// for its first rows, found without looking at the others' sizes beyond the sum before
// it; groups of more rows share those behind, so that one that gets all rows is spread
// over the chip too (6144 rows over 256 groups of 16 x 7168: 10.5 us with 24 rows each, 18.2
// with up to 406, 11.4 with all in one, and 10.5, 97 and 1419 where a workgroup went
// through all rows of its group).
#pragma once

#include "bst_mx4_gemm.hpp"

namespace bst {

template <int FM, int UNROLL, bool GROUPED>
struct Mx4Rows {
  static constexpr int NW = 8;

  // Loads have no branches around them, so that all of a step's are in flight
  // together: rows outside the matrix lie past the buffer's end, and a lane
  // without data gives an offset out of any range; both read zeros.
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), (short)0, (int)bytes, 0x00020000);
  }
  static __device__ __forceinline__ i32x4_t codes16(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t uniform_at,
                                                    bool in) {
    const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, in ? at : kOob, uniform_at, 0);
    return i32x4_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
  }
  // `left` of 32 codes are inside K; the rest may be anything and become zeros.
  static __device__ __forceinline__ void cut(i32x4_t& v, int left) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int n = left - 8 * d;
      v[d] &= n >= 8 ? -1 : n <= 0 ? 0 : (int)((1u << (4 * n)) - 1u);
    }
  }
  template <int S>
  static __device__ __forceinline__ f32x4_t product(const i32x4_t& x, const i32x4_t& y, const f32x4_t& c,
                                                    uint32_t sx, uint32_t sy) {
    const i32x8_t a = {x[0], x[1], x[2], x[3], 0, 0, 0, 0}, b = {y[0], y[1], y[2], y[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, S, (int)sx, S, (int)sy);
  }

  __device__ __attribute__((always_inline)) static void run(const Mx4GemmArgs& a) {
    __shared__ f32x4_t sums[FM][NW][64];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    // operand row; K 64q .. 64q + 63 of a block of 256: two chunks, two scale bytes
    const uint32_t r = lane & 15u, q = lane >> 4;
    uint32_t tile = blockIdx.x, g = 0, row0 = 0, rows = a.M;
    if constexpr (GROUPED) {
      const uint32_t tiles = (a.N + 15u) / 16u;
      g = tile / tiles;
      tile -= g * tiles;
      if (g < a.G) {
        // the group's first rows: sizes below 0 count as 0, and groups are cut to M rows
        int64_t before = 0;
        for (uint32_t i = lane; i < g; i += 64u) before += max(a.group_m[i], 0);
        for (int d = 32; d > 0; d >>= 1) before += __shfl_xor((long long)before, d);
        if (before >= (int64_t)a.M) return;
        row0 = __builtin_amdgcn_readfirstlane((uint32_t)before);
        rows = min((uint32_t)max(a.group_m[g], 0), a.M - row0);
      } else if (!later_rows(a, lane, g - a.G, g, row0, rows)) {
        return;
      }
      if (rows == 0) return;
    }
    const uint32_t n0 = tile * 16u, cols = min(a.N - n0, 16u);
    const uint32_t lda = (uint32_t)a.lda, ldb = (uint32_t)a.ldb, ldsa = (uint32_t)a.ldsa, ldsb = (uint32_t)a.ldsb;
    const uint32_t bo = r * ldb + 32 * q, so = r * ldsb + 2 * q;
    const __amdgpu_buffer_rsrc_t rb = buffer(a.B + (int64_t)g * a.strideB + (int64_t)n0 * a.ldb, cols * ldb),
                                 rsb = buffer(a.sb + (int64_t)g * a.strideSB + (int64_t)n0 * a.ldsb, cols * ldsb);
    const int64_t arow = row0;
    const uint32_t here = min(rows, 16u * FM);
    some_rows(a, sums, wave, lane, rb, rsb, buffer(a.A + arow * a.lda, here * lda),
              buffer(a.sa + arow * a.ldsa, here * ldsa), bo, so, lda, ldsa, arow, here, n0);
  }

  // The sum of x over the lanes up to this one.
  static __device__ __forceinline__ uint32_t sum_to_lane(uint32_t x) {
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xf, 0xf, false);  // 1, 2, 4 and 8 lanes
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xf, 0xf, false);  // back, in rows of 16
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xf, 0xf, false);
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xf, 0xf, false);
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xa, 0xf, false);  // a row's last to the next,
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xc, 0xf, false);  // the half's to the other
    return x;
  }

  // Part `want` of the groups' rows behind their first 16 FM, in the order of the
  // groups: its group, first row and the rows left from there.  False: there are not
  // so many.  Each lane has a group, 64 at a time; sizes above M count as M, so that
  // sums stay in 32 bits (M is at most 24 rows a group here).
  static __device__ __forceinline__ bool later_rows(const Mx4GemmArgs& a, uint32_t lane, uint32_t want, uint32_t& g,
                                                    uint32_t& row0, uint32_t& rows) {
    // (mostly there are none, and the launch waits for all its workgroups)
    uint64_t any = 0;
    for (uint32_t g0 = 0; g0 < a.G; g0 += 64u) any |= __ballot(g0 + lane < a.G && a.group_m[g0 + lane] > 16 * FM);
    if (any == 0) return false;
    uint32_t before = 0;  // rows of the groups before these 64
    for (uint32_t g0 = 0; g0 < a.G; g0 += 64u) {
      const uint32_t n = g0 + lane < a.G ? min((uint32_t)max(a.group_m[g0 + lane], 0), a.M) : 0u;
      const uint32_t end = before + sum_to_lane(n);
      const uint32_t lo = min(end - n, a.M), mine = min(end, a.M) - lo;
      const uint32_t parts = mine != 0 ? (mine - 1u) / (16u * FM) : 0u, last = sum_to_lane(parts);
      const uint64_t past = __ballot(last > want);
      if (past != 0) {
        const int at = __builtin_ctzll(past);
        const uint32_t skip = (1u + want - of_lane(last - parts, at)) * (16u * FM);
        g = g0 + (uint32_t)at;
        row0 = of_lane(lo, at) + skip;
        rows = of_lane(mine, at) - skip;
        return true;
      }
      before = of_lane(end, 63);
      want -= of_lane(last, 63);
    }
    return false;
  }
  static __device__ __forceinline__ uint32_t of_lane(uint32_t x, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
  }

  // Rows arow .. arow + here - 1 of A times the workgroup's columns.
  __device__ __attribute__((always_inline)) static void some_rows(
      const Mx4GemmArgs& a, f32x4_t (&sums)[FM][NW][64], uint32_t wave, uint32_t lane, __amdgpu_buffer_rsrc_t rb,
      __amdgpu_buffer_rsrc_t rsb, __amdgpu_buffer_rsrc_t ra, __amdgpu_buffer_rsrc_t rsa, uint32_t bo, uint32_t so,
      uint32_t lda, uint32_t ldsa, int64_t arow, uint32_t here, uint32_t n0) {
    const uint32_t r = lane & 15u, q = lane >> 4;
    f32x4_t acc[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t k0 = wave * UNROLL; k0 < a.nk; k0 += NW * UNROLL) {
      i32x4_t bv[UNROLL][2], av[UNROLL][FM][2];
      uint32_t sav[UNROLL][FM], sbv[UNROLL];
      auto left = [&](int u) {
        return k0 + u < a.nk ? (int)(a.K - (k0 + u) * kMx4Stage) - 64 * (int)q : 0;
      };
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const uint32_t at = (k0 + u) * 128u, sat = (k0 + u) * 8u;
        const int n = left(u);
#pragma unroll
        for (int s = 0; s < 2; ++s) bv[u][s] = codes16(rb, bo + 16 * s, at, n > 32 * s);
        sbv[u] = __builtin_amdgcn_raw_buffer_load_b16(rsb, n > 0 ? so : kOob, sat, 0);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const uint32_t row = i * 16 + r;
#pragma unroll
          for (int s = 0; s < 2; ++s) av[u][i][s] = codes16(ra, row * lda + 32 * q + 16 * s, at, n > 32 * s);
          sav[u][i] = __builtin_amdgcn_raw_buffer_load_b16(rsa, n > 0 ? row * ldsa + 2 * q : kOob, sat, 0);
        }
      }
      if ((a.K & 63u) != 0 && k0 + UNROLL >= a.nk) {
        // the last block: codes of A past K become zeros (so do the products), and so
        // do scale bytes past K, on both sides (a NaN scale times zero is not zero)
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          if (k0 + u + 1 != a.nk) continue;
          const int n = left(u);
          const uint32_t keep = n > 32 ? 0xffffu : 0xffu;
          sbv[u] &= keep;
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            sav[u][i] &= keep;
            cut(av[u][i][0], n);
            cut(av[u][i][1], n - 32);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u)
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          acc[i] = product<0>(bv[u][0], av[u][i][0], acc[i], sbv[u], sav[u][i]);
          acc[i] = product<1>(bv[u][1], av[u][i][1], acc[i], sbv[u], sav[u][i]);
        }
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) sums[i][wave][lane] = acc[i];
    __syncthreads();
    // wave w ends fragment w; lane l: row l & 15 of it, columns 4 (l >> 4) + 0..3
    if (wave >= (uint32_t)FM) return;
    f32x4_t s = sums[wave][0][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += sums[wave][w][lane];
    const uint32_t m = wave * 16 + r, c = n0 + 4 * q;
    if (m >= here || c >= a.N) return;
    const int64_t es = a.ckind == OUT_F32 ? 4 : 2;
    float v[4] = {s[0], s[1], s[2], s[3]};
    put_run<4>(a.C + ((arow + m) * a.ldc + c) * es, nullptr, v, a.N - c, a.cvec != 0 && a.N - c >= 4u, a.ckind);
  }
};

template <int FM, int UNROLL, bool GROUPED>
__global__ void __launch_bounds__(512) mx4_rows_kernel(Mx4GemmArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  Mx4Rows<FM, UNROLL, GROUPED>::run(a);
#endif
}

}  // namespace bst
