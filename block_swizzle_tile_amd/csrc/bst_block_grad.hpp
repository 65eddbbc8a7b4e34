// bst_block_grad.hpp -- the gradient of a linear layer's weight from its
// input kept in 8 bits:
//   dW[k][n] = add[k][n] + sum_m x[m][k] dY[m][n],  x[m][k] = q[m][k] 2^e[m][k/128].
//
// The sum runs over rows, and every row has its own scales, so they cannot
// leave the sum: x is restored on its way into LDS.  A code times a power of
// two is exact in bf16 (4 significant bits of 8; past the type's end it is the
// largest value, as bst_dequant_block gives it), one conversion instruction
// makes two of them, and each is made once per workgroup.  dY joins as bf16:
// as it is, or as 2 (fp16) or 3 (fp32) bf16 parts that add up to it, each
// with its own matrix product, so that nothing is rounded before the fp32
// sums.  Both operands lie in LDS row by row (m); the transposing reads turn
// 8 rows of a column into an operand of the 32x32x16 bf16 instruction.
//
// A stage's global loads are issued a whole step before they are converted and
// written to LDS, at the top of the step before the one that multiplies them.
#pragma once

#include "bst_block.hpp"

namespace bst {

struct BlockGradArgs {
  const uint8_t* Q;
  const uint8_t* S;
  const uint8_t* dY;
  const uint8_t* add;
  uint8_t* dW;
  int64_t ldq, lds, lddy, ldadd, lddw;  // elements
  int64_t strideadd, stridedw;
  const int32_t* group_m;               // null: one group of M rows
  float* part;                          // split > 1: [split][G][K][pitch]
  uint32_t pitch;
  uint32_t G, M, N, K;
  uint32_t tiles, tiles_all;            // per group, and G times that
  uint32_t split, remap, grid;
  uint32_t dwkind, dwvec, dyvec;
  MapConsts mc;                         // of one group's K x N tiles; core = tiles
};

enum DyKind { DY_BF16 = 0, DY_F16 = 1, DY_F32 = 2 };

// The bf16 part of f: f cut to bf16 (toward zero, so that no finite value
// becomes infinite); f then holds the rest, exactly.  An infinity or NaN is
// all in its first part.
__device__ __forceinline__ uint32_t take_part(float& f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f);
  uint32_t h = u & 0xffff0000u;
  if ((u & 0x7f800000u) == 0x7f800000u) {
    if (u & 0x007fffffu) h |= 0x00400000u;
    f = 0.0f;
  } else {
    f -= __builtin_bit_cast(float, h);
  }
  return h >> 16;
}

// Two bf16 whose infinities become the largest finite value, as when restoring:
// 256 * 2^120, the code of values within half a step of the type's end, is past
// it, and a zero gradient times an infinity would be NaN.  Only scale bytes of
// 247 and more reach that far.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
  w -= (w & 0x7fffu) == 0x7f80u ? 1u : 0u;
  return w - ((w & 0x7fff0000u) == 0x7f800000u ? 0x10000u : 0u);
}

template <int BK, int BN, int WM, int WN, int DY>
struct BlockGrad {
  static constexpr int NP = DY == DY_BF16 ? 1 : DY == DY_F16 ? 2 : 3;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int TM = BK / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  // rows per stage: two buffers of x and all parts of dY fit in LDS
  static constexpr int D = DY == DY_BF16 ? 64 : 32;
  static constexpr int XB = BK * 2, YB = BN * 2;  // bytes of an LDS row
  static constexpr int X_BYTES = D * XB, Y_BYTES = D * YB;
  static constexpr int STAGE_BYTES = X_BYTES + NP * Y_BYTES;
  static constexpr int XCH = BK / 16, YCH = BN / 8;  // loads per row: 16 codes, 8 gradients
  static constexpr int XL = D * XCH / NT, YL = D * YCH / NT;  // loads per thread
  static constexpr int KSTEPS = D / 16;

  static_assert(D * XCH % NT == 0 && D * YCH % NT == 0, "whole loads");
  static_assert(2 * STAGE_BYTES + (int)sizeof(RowGroups) <= 160 * 1024, "LDS budget");
  static_assert(NW * Strips<FM, FN>::BYTES <= 2 * STAGE_BYTES, "the epilogue's strips fit");

  static __device__ __forceinline__ lds_t* lds() {
    __shared__ __attribute__((aligned(16))) uint8_t buf[2 * STAGE_BYTES];
    return (lds_t*)buf;
  }
  template <int RB>
  static __device__ __forceinline__ uint32_t swz_r(uint32_t k) {
    return (((k & 1u) * 10u) + (((k >> 1) & 1u) * 4u)) & (uint32_t)(pow2_block(RB / 16) - 1);
  }

  // What a thread holds of the next stage.
  struct Held {
    u32x4_t x[XL];
    uint32_t e[XL];
    u32x4_t y[YL][DY == DY_F32 ? 2 : 1];
  };

  struct Src {
    const uint8_t *q, *s, *y;  // first row of the range, tile's first column
    int64_t ldq, lds, ldy;     // bytes
    uint32_t kcols, ncols;     // valid columns of the tile
    uint32_t rows;             // rows of the range
  };

  // Offsets of a thread's loads from the stage's first row; past the tile's
  // columns they are out of every buffer's range, and such loads give zeros.
  // (This runs on the host too, where a test checks every load.)
  struct Lanes {
    uint32_t x, e, y[DY == DY_F32 ? 2 : 1];
  };
  __host__ __device__ static __forceinline__ Lanes lanes(const Src& c, uint32_t tid) {
    const uint32_t xr = tid / XCH, xc = tid % XCH;
    const uint32_t yr = tid / YCH, yc = tid % YCH * 8;
    constexpr uint32_t ES = DY == DY_F32 ? 4 : 2, PER = 16 / ES;
    Lanes l;
    l.x = xc * 16 < c.kcols ? xr * (uint32_t)c.ldq + xc * 16 : kOob;
    l.e = xc * 16 < c.kcols ? xr * (uint32_t)c.lds + xc / 8 : kOob;
#pragma unroll
    for (uint32_t w = 0; w < (DY == DY_F32 ? 2 : 1); ++w)
      l.y[w] = yc + w * PER < c.ncols ? yr * (uint32_t)c.ldy + yc * ES + w * 16 : kOob;
    return l;
  }
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_from(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), (short)0, (int)kOob, 0x00020000);
  }

  // A stage's loads: no branches, so that they are all in flight together and
  // the conversion waits for each one by itself (with a branch around each, one
  // per bound, they were waited for together: 8192 x 4096 x 4096 266 us against
  // 239).  VEC: rows of dY start on 16 bytes.
  template <bool VEC>
  __device__ static __forceinline__ void load(Held& h, const Src& c, const Lanes& l, uint32_t r0) {
    constexpr uint32_t XR = NT / XCH, YR = NT / YCH;  // rows between a thread's loads
    const uint32_t left = r0 < c.rows ? c.rows - r0 : 0u;
    const int64_t at = left != 0 ? r0 : 0;
    const __amdgpu_buffer_rsrc_t q = rows_from(c.q + at * c.ldq), s = rows_from(c.s + at * c.lds);
#pragma unroll
    for (uint32_t i = 0; i < (uint32_t)XL; ++i) {
      const bool ok = i * XR + threadIdx.x / XCH < left;
      h.x[i] = __builtin_amdgcn_raw_buffer_load_b128(q, ok ? l.x : kOob, i * XR * (uint32_t)c.ldq, 0);
      h.e[i] = __builtin_amdgcn_raw_buffer_load_b8(s, ok ? l.e : kOob, i * XR * (uint32_t)c.lds, 0);
    }
    if constexpr (VEC) {
      const __amdgpu_buffer_rsrc_t y = rows_from(c.y + at * c.ldy);
#pragma unroll
      for (uint32_t i = 0; i < (uint32_t)YL; ++i) {
        const bool ok = i * YR + threadIdx.x / YCH < left;
#pragma unroll
        for (int w = 0; w < (DY == DY_F32 ? 2 : 1); ++w)
          h.y[i][w] = __builtin_amdgcn_raw_buffer_load_b128(y, ok ? l.y[w] : kOob,
                                                            i * YR * (uint32_t)c.ldy, 0);
      }
    } else {
      // rows that start anywhere: element by element
#pragma unroll
      for (uint32_t i = 0; i < (uint32_t)YL; ++i) {
        const uint32_t r = i * YR + threadIdx.x / YCH, n = threadIdx.x % YCH * 8;
#pragma unroll
        for (int w = 0; w < (DY == DY_F32 ? 2 : 1); ++w) h.y[i][w] = u32x4_t{0u, 0u, 0u, 0u};
        if (r >= left) continue;
        const uint8_t* p = c.y + (at + r) * c.ldy;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (n + e >= c.ncols) break;
          if constexpr (DY == DY_F32)
            h.y[i][e / 4][e % 4] = ((const uint32_t*)p)[n + e];
          else
            h.y[i][0][e / 2] |= (uint32_t)((const uint16_t*)p)[n + e] << (16 * (e & 1));
        }
      }
    }
  }

  __device__ static __forceinline__ void store(const Held& h, lds_t* base) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const uint32_t id = i * NT + threadIdx.x, r = id / XCH, ch = id % XCH;
      // the conversion reads only the exponent field: 0 is 2^-127, and 255 gives NaN
      const float s = __builtin_bit_cast(float, h.e[i] << 23);
      uint32_t o[8];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const b2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(h.x[i][d], s, false);
        const b2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(h.x[i][d], s, true);
        o[2 * d] = __builtin_bit_cast(uint32_t, lo);
        o[2 * d + 1] = __builtin_bit_cast(uint32_t, hi);
      }
      if (h.e[i] >= 247u) {
#pragma unroll
        for (int d = 0; d < 8; ++d) o[d] = finite_pair(o[d]);
      }
      lds_t* row = base + r * XB;
      const uint32_t z = swz_r<XB>(r);
      *(lds_u32x4_t*)(row + (((2 * ch) ^ z) << 4)) = u32x4_t{o[0], o[1], o[2], o[3]};
      *(lds_u32x4_t*)(row + (((2 * ch + 1) ^ z) << 4)) = u32x4_t{o[4], o[5], o[6], o[7]};
    }
#pragma unroll
    for (int i = 0; i < YL; ++i) {
      const uint32_t id = i * NT + threadIdx.x, r = id / YCH, ch = id % YCH;
      lds_t* at = base + X_BYTES + r * YB + ((ch ^ swz_r<YB>(r)) << 4);
      if constexpr (DY == DY_BF16) {
        *(lds_u32x4_t*)at = h.y[i][0];
      } else {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t w = h.y[i][DY == DY_F32 ? e / 4 : 0][DY == DY_F32 ? e % 4 : e / 2];
          if constexpr (DY == DY_F32)
            f[e] = __builtin_bit_cast(float, w);
          else
            f[e] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> (16 * (e & 1))));
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          u32x4_t o;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const uint32_t lo = take_part(f[2 * d]);
            o[d] = lo | take_part(f[2 * d + 1]) << 16;
          }
          *(lds_u32x4_t*)(at + p * Y_BYTES) = o;
        }
      }
    }
  }

  // 32 columns x 16 rows as an operand: lane l holds column col0 + (l & 31),
  // rows 16 kk + 8 (l >> 5) + 0..7.
  template <int RB>
  __device__ static __forceinline__ bf16x8_t frag(const lds_t* p, uint32_t col0, int kk,
                                                  uint32_t lane) {
    const uint32_t hi = lane >> 5, L = lane & 15u;
    const uint32_t colb = (col0 + 16 * ((lane >> 4) & 1u) + 4 * (L & 3u)) * 2;
    i16x4_t v[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t k = 16 * kk + 8 * hi + 4 * t + (L >> 2);
      v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_i16x4_t*)(p + k * RB + (((colb >> 4) ^ swz_r<RB>(k)) << 4) + (colb & 8u)));
    }
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
  }

  __device__ static __forceinline__ void compute(f32x16_t (&acc)[FM][FN], const lds_t* base,
                                                 uint32_t wm, uint32_t wn) {
    const uint32_t lane = threadIdx.x & 63u;
#pragma unroll
    for (int kk = 0; kk < KSTEPS; ++kk) {
      bf16x8_t x[FM], y[NP][FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) x[i] = frag<XB>(base, wm * TM + i * 32, kk, lane);
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          y[p][j] = frag<YB>(base + X_BYTES + p * Y_BYTES, wn * TN + j * 32, kk, lane);
#pragma unroll
      for (int p = NP - 1; p >= 0; --p)  // the small parts first
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y[p][j], x[i], acc[i][j], 0, 0, 0);
    }
  }

  template <bool VEC>
  __device__ static __forceinline__ void loop(f32x16_t (&acc)[FM][FN], const Src& c, uint32_t wm,
                                              uint32_t wn) {
    const Lanes l = lanes(c, threadIdx.x);
    Held h;
    load<VEC>(h, c, l, 0);
    store(h, lds());
    load<VEC>(h, c, l, D);
    uint32_t buf = 0;
    for (uint32_t r = 0; r < c.rows; r += D) {
      __syncthreads();  // buffer buf is written, and the other one read
      // loads past the last row read nothing
      if (r + D < c.rows) {
        store(h, lds() + (buf ^ 1u) * STAGE_BYTES);
        load<VEC>(h, c, l, r + 2 * D);
      }
      compute(acc, lds() + buf * STAGE_BYTES, wm, wn);
      buf ^= 1u;
    }
  }

  __device__ __attribute__((always_inline)) static void run(const BlockGradArgs& a) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t wm = wave / WN, wn = wave % WN;
    const uint32_t u = logical_wg(a.remap, a.grid);
    const uint32_t slice = a.mc.tiles.div(u);
    const uint32_t v = u - slice * a.tiles_all;
    const uint32_t g = a.mc.core.div(v);
    const TileCoord t = block_coord_fast(a.mc, v - g * a.tiles);
    // ---- rows of the group, then of this slice (whole stages)
    uint32_t row0 = 0, rows = a.M;
    if (a.group_m != nullptr) {
      __shared__ RowGroups groups;
      build_row_groups(groups, a.group_m, a.G, a.M, 1u, 1u);
      row0 = __builtin_amdgcn_readfirstlane(groups.first_row[g]);
      rows = __builtin_amdgcn_readfirstlane(groups.first_row[g + 1]) - row0;
    }
    const uint32_t stages = (rows + D - 1) / D;
    const uint32_t per = (stages + a.split - 1) / a.split * D;
    const uint32_t lo = slice * per < rows ? slice * per : rows;
    const uint32_t cnt = rows - lo < per ? rows - lo : per;
    const uint32_t k0 = t.m * BK, n0 = t.n * BN;
    constexpr int YES = DY == DY_F32 ? 4 : 2;
    Src c;
    const int64_t first = (int64_t)row0 + lo;
    c.ldq = a.ldq;
    c.lds = a.lds;
    c.ldy = a.lddy * YES;
    c.q = a.Q + first * c.ldq + k0;
    c.s = a.S + first * c.lds + k0 / kScaleBlock;
    c.y = a.dY + first * c.ldy + (int64_t)n0 * YES;
    c.kcols = a.K - k0 < (uint32_t)BK ? a.K - k0 : BK;
    c.ncols = a.N - n0 < (uint32_t)BN ? a.N - n0 : BN;
    c.rows = cnt;

    f32x16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    if (cnt > 0) {
      if (a.dyvec) loop<true>(acc, c, wm, wn);
      else loop<false>(acc, c, wm, wn);
      __syncthreads();
    }
    OutTile o;
    o.rows = c.kcols;
    o.cols = c.ncols;
    o.add = nullptr;
    o.ldadd_bytes = 0;
    if (a.part != nullptr) {
      o.kind = OUT_F32;
      o.vec = true;
      o.ld_bytes = (int64_t)a.pitch * 4;
      o.dst = (uint8_t*)(a.part + (((int64_t)slice * a.G + g) * a.K + k0) * a.pitch + n0);
    } else {
      o.kind = a.dwkind;
      o.vec = a.dwvec != 0;
      const int64_t es = a.dwkind == OUT_F32 ? 4 : 2;
      o.ld_bytes = a.lddw * es;
      o.dst = a.dW + (g * a.stridedw + (int64_t)k0 * a.lddw + n0) * es;
      if (a.add != nullptr) {
        o.ldadd_bytes = a.ldadd * es;
        o.add = a.add + (g * a.strideadd + (int64_t)k0 * a.ldadd + n0) * es;
      }
    }
    Strips<FM, FN>::template store<false>(lds() + wave * Strips<FM, FN>::BYTES, acc, wm * TM,
                                          wn * TN, o);
  }
};

template <int BK, int BN, int WM, int WN, int DY>
__global__ void __launch_bounds__(64 * WM * WN) block_grad_kernel(BlockGradArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  BlockGrad<BK, BN, WM, WN, DY>::run(a);
#endif
}

}  // namespace bst
