// bst_block_gemm.hpp -- the product of two e4m3 matrices with a scale per
// block of 128:
//   C[i][j] = sum_b sa[i][b] sb[b][j/128] sum_{k in block b} A[i][k] B[k][j].
//
// One pipeline stage is one scale block of K (128 bytes of every row), so the
// scales of a stage are one value per row of A and one value per wave of B (a
// wave's columns lie in one block of 128).  With E8M0 scales on both sides
// they are the scale operands of the matrix instruction and cost nothing.
// With 32-bit scales the instruction sums one block into a fresh accumulator
// and the vector unit adds it, scaled, to the running sum: the operands are
// swapped (B^T first), so a lane holds one row of C and its 16 columns share
// one factor sa * sb -- 16 fused multiply-adds per 128 matrix-pipe cycles.
#pragma once

#include "bst_block.hpp"

namespace bst {

struct BlockGemmArgs {
  const uint8_t* A;
  const uint8_t* B;
  uint8_t* C;
  const uint8_t* sa;
  const uint8_t* sb;
  int64_t lda, ldb, ldc, ldsa, ldsb;  // elements
  int64_t strideB, strideSB;          // grouped: elements per group
  const int32_t* group_m;
  float* part;                        // split > 1: [split][M][pitch] partial sums
  uint32_t pitch;
  uint32_t G, M, N, K;                // M: total rows when grouped
  uint32_t nk, kslice;                // stages in all and per slice
  uint32_t tiles;                     // plain: tasks per slice
  uint32_t off, dir, remap, grid;
  uint32_t sa_f32, sb_f32;            // scale types
  uint32_t ckind, cvec;
  MapConsts mc;
};

// How a stage's products are formed and scaled (see above).
enum BlockMode { MODE_E8M0 = 0, MODE_F32 = 1, MODE_EXACT = 2 };

// One byte per lane, zero-extended to a dword of LDS.
__device__ __forceinline__ void dma1(const u32x4_t& desc, const lds_t* lds, uint32_t voff) {
  asm volatile("s_nop 4\n\tbuffer_load_ubyte %1, %2, 0 offen lds"
               :
               : "{m0}"((uint32_t)(uintptr_t)lds), "v"(voff), "s"(uniform(desc))
               : "memory");
}

template <int BM, int BN, int WM, int WN, int STAGES, bool TB, int MODE, bool GROUPED>
struct BlockGemm {
  static constexpr bool HW = MODE == MODE_E8M0;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int A_IPW = A_BYTES / 1024 / NW, B_IPW = B_BYTES / 1024 / NW;
  static constexpr int NCH = BN / 16;  // 16-byte chunks of a K row of B (TB = 0)
  static constexpr uint32_t BSWZ = pow2_block(NCH) - 1;
  // A's scales: one dword per row, 64 rows per instruction, one instruction
  // per wave at most; waves past them load nothing into a spare area, so
  // that every wave has the same count in flight
  static constexpr int SA_N = (BM + 63) / 64;
  static constexpr int SA_BYTES = SA_N * 256;
  static constexpr int SPARE = SA_N < NW ? 256 : 0;
  static constexpr int LPS = A_IPW + B_IPW + 1;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SA_BYTES + SPARE;
  static constexpr int LDS_BYTES = STAGES * STAGE_BYTES;

  static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0, "whole DMA waves");
  static_assert(SA_N <= NW, "one scale instruction per wave");
  static_assert(TM % 32 == 0 && TN % 32 == 0 && 128 % TN == 0, "wave tile");
  static_assert(NW * Strip<TN>::BYTES <= LDS_BYTES, "the epilogue's strips fit");
  static_assert((STAGES - 1) * LPS < 64, "vmcnt holds 6 bits");
  static_assert(LDS_BYTES + (GROUPED ? (int)sizeof(RowGroups) : 0) <= 160 * 1024, "LDS budget");

  static __device__ __forceinline__ lds_t* lds() {
    __shared__ __attribute__((aligned(16))) uint8_t buf[LDS_BYTES];
    return (lds_t*)buf;
  }
  static __device__ __forceinline__ uint32_t swz_b(uint32_t k) {
    return ((k & 7u) + (k & 1u) * 8u) & BSWZ;
  }

  template <int N>
  __device__ static __forceinline__ void wait_vm() {
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  }

  struct Lanes {
    uint32_t a_off[A_IPW], b_off[B_IPW];  // byte offset in the stage's panel, or kOob
    uint32_t a_k[A_IPW], b_k[B_IPW];      // K index of the access inside the stage
    uint32_t s_off;
  };

  struct Src {
    const uint8_t *a, *b, *sa;  // panels of the task at K = 0
    int64_t ldb;
    uint32_t K, sa_f32, wave;
  };

  // DMA of stage kt (K rows kt*128 ..) into buffer s.  Accesses at or past K
  // are sent out of the descriptor's range and write zeros.
  __device__ static __forceinline__ void issue(const Src& c, const Lanes& ln, uint32_t kt,
                                               uint32_t s) {
    lds_t* base = lds() + s * STAGE_BYTES;
    const uint32_t left = c.K - kt * 128u;
    const u32x4_t ra = make_desc(c.a + (uint64_t)kt * 128u);
    const u32x4_t rb = make_desc(c.b + (TB ? (int64_t)kt * 128 : (int64_t)kt * 128 * c.ldb));
#pragma unroll
    for (int i = 0; i < A_IPW; ++i)
      dma16(ra, base + (c.wave * A_IPW + i) * 1024, ln.a_k[i] < left ? ln.a_off[i] : kOob, 0u);
#pragma unroll
    for (int i = 0; i < B_IPW; ++i)
      dma16(rb, base + A_BYTES + (c.wave * B_IPW + i) * 1024,
            ln.b_k[i] < left ? ln.b_off[i] : kOob, 0u);
    lds_t* sdst = base + A_BYTES + B_BYTES + (c.wave < (uint32_t)SA_N ? c.wave * 256u : SA_BYTES);
    if (c.sa_f32)
      dma4(make_desc(c.sa + (uint64_t)kt * 4u), sdst, ln.s_off, 0u);
    else
      dma1(make_desc(c.sa + kt), sdst, ln.s_off);
  }

  // K % 16 != 0: the last chunk of a row holds bytes past K, which may be
  // anything (a NaN code times a zero is not zero).  They are cleared in LDS
  // after the stage has landed.
  __device__ static __forceinline__ void clear_tail(lds_t* base, uint32_t k_in_stage) {
    const uint32_t c = k_in_stage >> 4, keep = k_in_stage & 15u;
    for (uint32_t r = threadIdx.x; r < (uint32_t)(BM + (TB ? BN : 0)); r += NT) {
      const uint32_t row = r < (uint32_t)BM ? r : r - BM;
      lds_t* p = base + (r < (uint32_t)BM ? 0 : A_BYTES) + lds_off(row, c);
      u32x4_t v = *(const lds_u32x4_t*)p;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int n = (int)keep - 4 * d;  // bytes of this dword to keep
        v[d] = n >= 4 ? v[d] : n <= 0 ? 0u : v[d] & ((1u << (8 * n)) - 1u);
      }
      *(lds_u32x4_t*)p = v;
    }
    __syncthreads();
  }

  __device__ static __forceinline__ i32x8_t rows_frag(const lds_t* base, uint32_t row, int kk,
                                                      uint32_t hi) {
    const lds_t* rp = base + row * 128;
    const u32x4_t x = *(const lds_u32x4_t*)(rp + (((4 * kk + hi) ^ swz(row)) << 4));
    const u32x4_t y = *(const lds_u32x4_t*)(rp + (((4 * kk + 2 + hi) ^ swz(row)) << 4));
    return i32x8_t{(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                   (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  }

  // B fragment from K rows: four transposing reads (8 K values each) in the
  // K order of rows_frag.
  __device__ static __forceinline__ i32x8_t cols_frag(const lds_t* lb, uint32_t col0, int kk,
                                                      uint32_t lane) {
    const uint32_t hi = lane >> 5, L = lane & 15u;
    const uint32_t colb = col0 + 16 * ((lane >> 4) & 1u) + 8 * (L & 1u);
    i32x2_t v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t k = 64 * kk + 32 * (t >> 1) + 16 * hi + 8 * (t & 1) + (L >> 1);
      v[t] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (lds_i32x2_t*)(lb + k * BN + (((colb >> 4) ^ swz_b(k)) << 4) + (colb & 8u)));
    }
    return i32x8_t{v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]};
  }

  // Codes of a fragment's bytes 8s .. 8s+7 as a bf16 operand.
  __device__ static __forceinline__ bf16x8_t widen(const i32x8_t& f, int s) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    u32x4_t o;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const uint32_t w = (uint32_t)f[2 * s + d];
      o[2 * d] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
      o[2 * d + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
    }
    return __builtin_bit_cast(bf16x8_t, o);
  }

  // The products of one stage.
  __device__ static __forceinline__ void compute(f32x16_t (&acc)[FM][FN], const lds_t* base,
                                                 uint32_t wm, uint32_t wn, uint32_t sb_raw,
                                                 bool sa_f32, bool sb_f32) {
    const uint32_t lane = threadIdx.x & 63u, l32 = lane & 31u, hi = lane >> 5;
    const lds_t* lb = base + A_BYTES;
    auto a_frag = [&](int i, int kk) { return rows_frag(base, wm * TM + i * 32 + l32, kk, hi); };
    auto b_frag = [&](int j, int kk) {
      if constexpr (TB)
        return rows_frag(lb, wn * TN + j * 32 + l32, kk, hi);
      else
        return cols_frag(lb, wn * TN + j * 32, kk, lane);
    };
    uint32_t sa[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
      sa[i] = *(const lds_u32_t*)(lb + B_BYTES + (wm * TM + i * 32 + l32) * 4);
    if constexpr (HW) {
      const uint32_t sb = sb_raw & 0xffu;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        i32x8_t a[FM], b[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) a[i] = a_frag(i, kk);
#pragma unroll
        for (int j = 0; j < FN; ++j) b[j] = b_frag(j, kk);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                b[j], a[i], acc[i][j], 0, 0, 0, (int)sb, 0, (int)sa[i]);
      }
    } else {
      const float fb = sb_f32 ? __builtin_bit_cast(float, sb_raw) : e8m0_value(sb_raw & 0xffu);
      i32x8_t b[2][FN];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int j = 0; j < FN; ++j) b[kk][j] = b_frag(j, kk);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const float f = (sa_f32 ? __builtin_bit_cast(float, sa[i]) : e8m0_value(sa[i])) * fb;
        const i32x8_t a[2] = {a_frag(i, 0), a_frag(i, 1)};
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          f32x16_t p = {};
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            if constexpr (MODE == MODE_EXACT) {
#pragma unroll
              for (int s = 0; s < 4; ++s)
                p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen(b[kk][j], s), widen(a[kk], s), p,
                                                            0, 0, 0);
            } else {
              p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[kk][j], a[kk], p, 0, 0, 0, 0x7f,
                                                                  0, 0x7f);
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][j][e] = __builtin_fmaf(f, p[e], acc[i][j][e]);
        }
      }
    }
  }

  __device__ __attribute__((always_inline)) static void run(const BlockGemmArgs& a) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wm = wave / WN, wn = wave % WN;
    // ---- the task: tile (m, n) of a group or of a K slice
    uint32_t g = 0, row0 = 0, rows = a.M, slice = 0;
    TileCoord t;
    if constexpr (GROUPED) {
      __shared__ RowGroups groups;
      const uint32_t loops_n = (a.N + BN - 1) / BN;
      build_row_groups(groups, a.group_m, a.G, a.M, BM, loops_n);
      const uint32_t T = groups.first_task[a.G];
      if (blockIdx.x >= T) return;  // the whole workgroup
      const uint32_t u = logical_wg(a.remap, T);
      uint32_t lo = 0, hi = a.G - 1;  // the last group whose first task is <= u
      while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) >> 1;
        if (groups.first_task[mid] <= u) lo = mid; else hi = mid - 1;
      }
      g = __builtin_amdgcn_readfirstlane(lo);
      row0 = __builtin_amdgcn_readfirstlane(groups.first_row[g]);
      rows = __builtin_amdgcn_readfirstlane(groups.first_row[g + 1]) - row0;
      const uint32_t inner = __builtin_amdgcn_readfirstlane(u - groups.first_task[g]);
      t = block_coord((rows + BM - 1) / BM, loops_n, a.off, a.dir, inner);
    } else {
      const uint32_t u = logical_wg(a.remap, a.grid);
      slice = a.mc.tiles.div(u);
      t = block_coord_fast(a.mc, u - slice * a.tiles);
    }
    const uint32_t m0 = t.m * BM, n0 = t.n * BN;
    const uint32_t rows_left = rows - m0 < (uint32_t)BM ? rows - m0 : BM;
    const uint32_t cols_left = a.N - n0 < (uint32_t)BN ? a.N - n0 : BN;
    const uint32_t kt0 = slice * a.kslice;
    const uint32_t kt1 = a.nk - kt0 < a.kslice ? a.nk : kt0 + a.kslice;
    // ---- its panels
    const int64_t arow = (int64_t)row0 + m0;
    Src c;
    c.a = a.A + arow * a.lda;
    c.b = a.B + (int64_t)g * a.strideB + (TB ? (int64_t)n0 * a.ldb : (int64_t)n0);
    c.sa_f32 = HW ? 0u : a.sa_f32;
    c.sa = a.sa + arow * a.ldsa * (c.sa_f32 ? 4 : 1);
    c.ldb = a.ldb;
    c.K = a.K;
    c.wave = wave;
    // the block column of this wave's columns (kept inside N for waves past it)
    const uint32_t wcol = n0 + wn * TN < a.N ? n0 + wn * TN : a.N - 1;
    const bool sb_f32 = !HW && a.sb_f32;
    const int64_t sb_step = (TB ? 1 : a.ldsb) * (sb_f32 ? 4 : 1);
    const uint8_t* sb = a.sb + ((int64_t)g * a.strideSB +
                                (int64_t)(wcol / kScaleBlock) * (TB ? a.ldsb : 1)) *
                                   (sb_f32 ? 4 : 1);
    Lanes ln;
#pragma unroll
    for (int i = 0; i < A_IPW; ++i) {
      const uint32_t r = (wave * A_IPW + i) * 8 + (lane >> 3), ch = (lane & 7u) ^ swz(r);
      ln.a_k[i] = ch * 16;
      ln.a_off[i] = r < rows_left ? r * (uint32_t)a.lda + ch * 16 : kOob;
    }
#pragma unroll
    for (int i = 0; i < B_IPW; ++i) {
      if constexpr (TB) {
        const uint32_t r = (wave * B_IPW + i) * 8 + (lane >> 3), ch = (lane & 7u) ^ swz(r);
        ln.b_k[i] = ch * 16;
        ln.b_off[i] = r < cols_left ? r * (uint32_t)a.ldb + ch * 16 : kOob;
      } else {
        const uint32_t byte = (wave * B_IPW + i) * 1024 + lane * 16;
        const uint32_t k = byte / BN, ch = ((byte % BN) / 16) ^ swz_b(k);
        ln.b_k[i] = k;
        ln.b_off[i] = ch * 16 < cols_left ? k * (uint32_t)a.ldb + ch * 16 : kOob;
      }
    }
    const uint32_t srow = wave * 64 + lane;
    ln.s_off = wave < (uint32_t)SA_N && srow < rows_left
                   ? srow * (uint32_t)a.ldsa * (c.sa_f32 ? 4u : 1u) : kOob;

    f32x16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    // ---- K loop: at the top of a step stage kt must have landed and the
    // STAGES - 2 stages behind it may still be in flight
    for (uint32_t s = 0; s < (uint32_t)STAGES - 1; ++s)
      if (kt0 + s < kt1) issue(c, ln, kt0 + s, s);
    uint32_t buf = 0;
    uint32_t sb_raw = kt0 < kt1 ? scalar_dword(sb + kt0 * sb_step) : 0u;
    for (uint32_t kt = kt0; kt < kt1; ++kt) {
      if (kt + STAGES - 1 <= kt1) wait_vm<(STAGES - 2) * LPS>(); else wait_vm<0>();
      barrier_lds();
      const uint32_t nb = buf == 0 ? STAGES - 1 : buf - 1;  // the buffer read in the last step
      if (kt + STAGES - 1 < kt1) issue(c, ln, kt + STAGES - 1, nb);
      const uint32_t sb_now = sb_raw;
      if (kt + 1 < kt1) sb_raw = scalar_dword(sb + (kt + 1) * sb_step);
      lds_t* base = lds() + buf * STAGE_BYTES;
      if (kt + 1 == a.nk && (a.K & 15u)) clear_tail(base, a.K & 127u);
      compute(acc, base, wm, wn, sb_now, c.sa_f32 != 0, sb_f32);
      buf = buf + 1 == STAGES ? 0 : buf + 1;
    }
    // ---- every wave is done with the stages: their LDS holds the strips
    __builtin_amdgcn_s_waitcnt(0);
    barrier_lds();
    OutTile o;
    o.add = nullptr;
    o.ldadd_bytes = 0;
    o.rows = rows_left;
    o.cols = cols_left;
    if (!GROUPED && a.part != nullptr) {
      o.kind = OUT_F32;
      o.vec = true;
      o.ld_bytes = (int64_t)a.pitch * 4;
      o.dst = (uint8_t*)(a.part + ((int64_t)slice * a.M + m0) * a.pitch + n0);
    } else {
      o.kind = a.ckind;
      o.vec = a.cvec != 0;
      const int64_t es = a.ckind == OUT_F32 ? 4 : 2;
      o.ld_bytes = a.ldc * es;
      o.dst = a.C + (arow * a.ldc + n0) * es;
    }
    store_wave_tile<FM, FN>(lds() + wave * Strip<TN>::BYTES, acc, wm * TM, wn * TN, o);
  }
};

template <int BM, int BN, int WM, int WN, int STAGES, bool TB, int MODE, bool GROUPED>
__global__ void __launch_bounds__(64 * WM * WN) block_gemm_kernel(BlockGemmArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  BlockGemm<BM, BN, WM, WN, STAGES, TB, MODE, GROUPED>::run(a);
#endif
}

}  // namespace bst
