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

// Codes of a fragment's bytes 8s .. 8s+7 as a bf16 operand.
__device__ __forceinline__ bf16x8_t widen_codes(const i32x8_t& f, int s) {
  u32x4_t o;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const uint32_t w = (uint32_t)f[2 * s + d];
    o[2 * d] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    o[2 * d + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
  }
  return __builtin_bit_cast(bf16x8_t, o);
}

template <int BM, int BN, int WM, int WN, int STAGES, bool TB, int MODE, bool GROUPED>
struct BlockGemm {
  static constexpr bool HW = MODE == MODE_E8M0;
  static constexpr bool RING = STAGES >= 3;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int A_IPW = A_BYTES / 1024 / NW, B_IPW = B_BYTES / 1024 / NW;
  static constexpr int NCH = BN / 16;  // 16-byte chunks of a K row of B (TB = 0)
  static constexpr uint32_t BSWZ = pow2_block(NCH) - 1;
  // Scales ride with the stage, one DMA instruction per wave: waves below
  // SA_N take A's (a dword per row, 64 rows each), wave SA_N takes B's (a
  // dword per block of columns), and any further waves load nothing into a
  // spare area, so that every wave has the same count in flight.  (Scalar
  // loads of B's scale share a counter with the LDS reads, which then wait for
  // their cache misses: 64 rows over 16 K x N weights of 4096 x 2048 30.4 us,
  // with the DMA 22.6.)
  static constexpr int SA_N = (BM + 63) / 64;
  static constexpr int SA_BYTES = SA_N * 256;
  static constexpr int SB_BYTES = 256;
  static constexpr int SPARE = SA_N + 1 < NW ? 256 : 0;
  static constexpr int LPS = A_IPW + B_IPW + 1;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES + SPARE;
  static constexpr int LDS_BYTES = STAGES * STAGE_BYTES;

  static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0, "whole DMA waves");
  static_assert(SA_N < NW, "one scale instruction per wave");
  static_assert(RING || MODE != MODE_EXACT, "the two-stage loop has no exact form");
  static_assert(TM % 32 == 0 && TN % 32 == 0 && 128 % TN == 0, "wave tile");
  static_assert(NW * Strips<FM, FN>::BYTES <= LDS_BYTES, "the epilogue's strips fit");
  static_assert((STAGES - 1) * LPS < 64, "vmcnt holds 6 bits");
  static_assert(LDS_BYTES + (GROUPED ? (int)sizeof(RowGroups) : 0) <= 160 * 1024, "LDS budget");

  static __device__ __forceinline__ lds_t* lds() {
    __shared__ __attribute__((aligned(16))) uint8_t buf[LDS_BYTES];
    return (lds_t*)buf;
  }
  static __host__ __device__ __forceinline__ uint32_t swz_b(uint32_t k) {
    return ((k & 7u) + (k & 1u) * 8u) & BSWZ;
  }

  template <int N>
  __device__ static __forceinline__ void wait_vm() {
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  }

  // A lane's part of the DMA addressing.  Instruction x of a wave covers 8
  // rows of A (or of a transposed B), or RPB K rows of B; the lane's offset
  // is its offset in the wave's first rows with the chunk index exchanged by
  // an XOR that only depends on the instruction, and the rows go to the scalar
  // offset: two registers hold what a register per instruction would (those
  // did not fit beside the accumulators of the 256 x 256 tile).
  struct Lanes {
    uint32_t a_row, b_row;  // offset of the lane's row in an instruction's rows
    uint32_t a_ch, b_ch;    // its chunk, before the instruction's XOR
    uint32_t inside;        // bit x: access x is inside the matrix (rows; columns of B)
    uint32_t tail;          // bit x: and inside K in the last, partial stage
    uint32_t s_off;
  };
  static constexpr int RPB = TB ? 8 : 1024 / BN;
  // instruction x of wave w: its XOR and its first row (or K row)
  static __host__ __device__ __forceinline__ uint32_t a_xor(uint32_t w, int x) {
    return (w * A_IPW + x) & 7u;
  }
  static __host__ __device__ __forceinline__ uint32_t b_xor(uint32_t w, int x) {
    return TB ? (w * B_IPW + x) & 7u : ((w * B_IPW + x) * RPB) & 7u & BSWZ;
  }

  // What the addressing needs of a tile.  (It runs on the host too, where a test
  // checks every access.)
  struct Tile {
    uint32_t lda32, ldb32, K;
    uint32_t rows_left, cols_left;  // valid rows and columns
    uint32_t s_pitch;  // bytes between the wave's scales: of two rows of A, or two blocks of columns
    uint32_t blocks;   // blocks of columns from the tile's first on
  };
  static __host__ __device__ __forceinline__ Lanes lanes(const Tile& t, uint32_t wave, uint32_t lane) {
    Lanes ln;
    const uint32_t last = t.K & 127u;      // K rows of a partial last stage
    constexpr int LPR = TB ? 8 : BN / 16;  // lanes per row of B
    ln.a_row = (lane >> 3) * t.lda32;
    ln.a_ch = (lane & 7u) ^ (lane >> 3);
    ln.b_row = (lane / LPR) * t.ldb32;
    ln.b_ch = (lane % LPR) ^ (TB ? lane >> 3 : swz_b(lane / LPR));
    ln.inside = ln.tail = 0;
#pragma unroll
    for (int x = 0; x < A_IPW; ++x) {
      const uint32_t r = (wave * A_IPW + x) * 8 + (lane >> 3), ch = ln.a_ch ^ a_xor(wave, x);
      if (r < t.rows_left) ln.inside |= 1u << x;
      if (r < t.rows_left && ch * 16 < last) ln.tail |= 1u << x;
    }
#pragma unroll
    for (int x = 0; x < B_IPW; ++x) {
      const uint32_t r = (wave * B_IPW + x) * RPB + lane / LPR, ch = ln.b_ch ^ b_xor(wave, x);
      const uint32_t k = TB ? ch * 16 : r;
      const bool in = TB ? r < t.cols_left : ch * 16 < t.cols_left;
      if (in) ln.inside |= 1u << (A_IPW + x);
      if (in && k < last) ln.tail |= 1u << (A_IPW + x);
    }
    if (wave < (uint32_t)SA_N)
      ln.s_off = wave * 64 + lane < t.rows_left ? (wave * 64 + lane) * t.s_pitch : kOob;
    else
      ln.s_off = wave == (uint32_t)SA_N && lane < (BN + 127) / 128 && lane < t.blocks
                     ? lane * t.s_pitch : kOob;
    return ln;
  }
  // Bit x: access x of a lane is inside its matrix in stage kt of a slice that ends at kt1.
  static __host__ __device__ __forceinline__ uint32_t live(const Lanes& ln, uint32_t kt, uint32_t kt1,
                                                           uint32_t K) {
    return kt >= kt1 ? 0u : (kt + 1) * 128u <= K ? ln.inside : ln.tail;
  }
  // Access X of a wave's lane: 16 bytes at lane + wave offset of A's panel (X <
  // A_IPW) or B's, and where the wave's 1024 bytes go in the stage's LDS.
  struct Access {
    uint32_t voff, soff, lds;
  };
  template <int X>
  static __host__ __device__ __forceinline__ Access access(uint32_t wave, uint32_t lda32, uint32_t ldb32,
                                                           const Lanes& ln, uint32_t live_bits,
                                                           uint32_t a_ch, uint32_t b_ch) {
    if constexpr (X < A_IPW) {
      const uint32_t off = ln.a_row + ((a_ch ^ a_xor(wave, X)) << 4);
      return Access{(live_bits >> X) & 1u ? off : kOob, (wave * A_IPW + X) * 8 * lda32,
                    (wave * A_IPW + X) * 1024};
    } else {
      constexpr int x = X - A_IPW;
      const uint32_t off = ln.b_row + ((b_ch ^ b_xor(wave, x)) << 4);
      return Access{(live_bits >> X) & 1u ? off : kOob, (wave * B_IPW + x) * RPB * ldb32,
                    (uint32_t)A_BYTES + (wave * B_IPW + x) * 1024};
    }
  }

  struct Src {
    const uint8_t *a, *b;  // panels of the task at K = 0
    const uint8_t* s;      // the scales this wave loads, at K = 0
    int64_t ldb, s_step;   // s_step: bytes from one K block's scales to the next's
    uint32_t lda32, ldb32;
    uint32_t K, kt1, s_f32, wave;
  };

  // Where one stage's DMA reads and writes.
  struct Stage {
    u32x4_t ra, rb;
    lds_t* base;
    uint32_t live;  // bit x: this lane's access x is inside its matrix
    uint32_t a_ch, b_ch;
  };

  // Stage kt (K rows kt*128 ..) into buffer s.  A stage past the slice's last
  // is issued all the same, with every access out of range: the counts in
  // flight then never depend on where the loop is, and what it writes (zeros)
  // is never read.
  __device__ static __forceinline__ Stage stage(const Src& c, const Lanes& ln, uint32_t kt,
                                                uint32_t s) {
    Stage st;
    st.ra = make_desc(c.a + (uint64_t)kt * 128u);
    st.rb = make_desc(c.b + (TB ? (int64_t)kt * 128 : (int64_t)kt * 128 * c.ldb));
    st.base = lds() + s * STAGE_BYTES;
    st.a_ch = fresh_v(ln.a_ch);  // offsets are made anew for every stage, not kept
    st.b_ch = fresh_v(ln.b_ch);
    st.live = live(ln, kt, c.kt1, c.K);
    return st;
  }
  static constexpr int ND = A_IPW + B_IPW;
  template <int X>
  __device__ static __forceinline__ void dma_one(const Src& c, const Lanes& ln, const Stage& st) {
    const Access m = access<X>(c.wave, c.lda32, c.ldb32, ln, st.live, st.a_ch, st.b_ch);
    dma16(X < A_IPW ? st.ra : st.rb, st.base + m.lds, m.voff, m.soff);
  }
  __device__ static __forceinline__ void dma_scales(const Src& c, const Lanes& ln, const Stage& st,
                                                    uint32_t kt) {
    // A's areas, B's and the spare one follow each other in wave order
    constexpr uint32_t spare = SPARE ? SA_N + 1 : SA_N;
    lds_t* dst = st.base + A_BYTES + B_BYTES + (c.wave < spare ? c.wave : spare) * 256u;
    const uint32_t v = kt < c.kt1 ? ln.s_off : kOob;
    const u32x4_t d = make_desc(c.s + (int64_t)kt * c.s_step);
    if (c.s_f32)
      dma4(d, dst, v, 0u);
    else
      dma1(d, dst, v);
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

  // Operand fragments: lane l holds row (l & 31) of a 32-row fragment, K =
  // 64 kk + 16 (l >> 5) + 0..15 and 32 more.  Rows of 128 bytes with their
  // chunks XORed by swz(row): fragment i of a wave lies 32 i rows on, which
  // only flips bit 2 of the XOR for odd i, so four lane addresses (two chunks,
  // plain and flipped) serve all of them with constant offsets.
  struct RowPtrs {
    const lds_t* p[4];
  };
  __device__ static __forceinline__ RowPtrs row_ptrs(const lds_t* base, uint32_t row0) {
    const uint32_t lane = threadIdx.x & 63u, row = row0 + (lane & 31u), hi = lane >> 5;
    RowPtrs r;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      r.p[v] = base + row * 128 + ((((v & 1) * 2 + hi) ^ swz(row) ^ ((v >> 1) * 4u)) << 4);
    return r;
  }
  __device__ static __forceinline__ i32x8_t rows_frag(const RowPtrs& r, int i, int kk) {
    const int s = 2 * (kk ^ (i & 1));
    const u32x4_t x = *(const lds_u32x4_t*)(r.p[s] + i * 4096);
    const u32x4_t y = *(const lds_u32x4_t*)(r.p[s + 1] + i * 4096);
    return i32x8_t{(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                   (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  }

  // B fragment from K rows: four transposing reads (8 K values each) in the
  // K order of rows_frag.  A lane's K rows differ by multiples of 8, which
  // leave the XOR of the columns' chunk alone, and fragment j flips bit 1 of
  // the chunk: one address per j.
  struct ColPtrs {
    const lds_t* p[FN];
  };
  __device__ static __forceinline__ ColPtrs col_ptrs(const lds_t* lb, uint32_t wn) {
    const uint32_t lane = threadIdx.x & 63u, hi = lane >> 5, L = lane & 15u;
    const uint32_t k = 16 * hi + (L >> 1);
    const uint32_t ch = (wn * TN) / 16 + ((lane >> 4) & 1u);
    ColPtrs r;
#pragma unroll
    for (int j = 0; j < FN; ++j)
      r.p[j] = lb + k * BN + (((ch ^ (2u * j)) ^ swz_b(k)) << 4) + 8 * (L & 1u);
    return r;
  }
  __device__ static __forceinline__ i32x8_t cols_frag(const ColPtrs& r, int j, int kk) {
    i32x2_t v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      v[t] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (lds_i32x2_t*)(r.p[j] + (64 * kk + 32 * (t >> 1) + 8 * (t & 1)) * BN));
    return i32x8_t{v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]};
  }

  // The products of one stage of the 256x256 tile, whose registers leave no
  // room for a second set of operands (its fp32 outputs none for widened
  // ones), with the DMA of the next stage between them.  The order is fixed by hand, one matrix instruction per slot:
  // behind each go its share of the DMA instructions (one per slot from the
  // first: with two stages they have only this step to land in), the LDS
  // reads of the operands that the slots ahead need, and with 32-bit scales
  // half of the 16 multiply-adds of the sub-tile before, which the vector unit
  // does while the matrix unit works on this one.
  __device__ static __forceinline__ void compute(f32x16_t (&acc)[FM][FN], const lds_t* base,
                                                 uint32_t wm, uint32_t wn, bool sa_f32, bool sb_f32,
                                                 const Src& c, const Lanes& ln,
                                                 const Stage& next) {
    const uint32_t l32 = threadIdx.x & 31u;
    const lds_t* lb = base + A_BYTES;
    const RowPtrs pa = row_ptrs(base, wm * TM);
    const auto pb = [&] {
      if constexpr (TB) return row_ptrs(lb, wn * TN);
      else return col_ptrs(lb, wn);
    }();
    auto a_frag = [&](int i, int kk) { return rows_frag(pa, i, kk); };
    auto b_frag = [&](int j, int kk) {
      if constexpr (TB) return rows_frag(pb, j, kk);
      else return cols_frag(pb, j, kk);
    };
    constexpr int NS = 2 * FM * FN;           // slots
    constexpr int DS = NS < ND ? NS : ND;     // slots that carry DMA
    auto slot_dma = [&](auto q) {
      constexpr int Q = decltype(q)::value;
      if constexpr (Q < DS)
        static_for_range<Q * ND / DS, (Q + 1) * ND / DS>(
            [&](auto x) { dma_one<decltype(x)::value>(c, ln, next); });
    };
    uint32_t sa[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
      sa[i] = *(const lds_u32_t*)(lb + B_BYTES + (wm * TM + i * 32 + l32) * 4);
    // the block of this wave's columns: the tile starts inside a block only
    // if it is narrower than one, and then holds one
    const uint32_t sb_raw = *(const lds_u32_t*)(lb + B_BYTES + SA_BYTES + (wn * TN / kScaleBlock) * 4);
    if constexpr (HW) {
      const uint32_t sb = sb_raw;
      i32x8_t a[2][FM], b[2][FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) b[0][j] = b_frag(j, 0);
#pragma unroll
      for (int i = 0; i < FM; ++i) a[0][i] = a_frag(i, 0);
      static_for<NS>([&](auto q) {
        constexpr int Q = decltype(q)::value, NM = FM * FN, NL = FM + FN;
        constexpr int kk = Q / NM, R = Q % NM, i = R / FN, j = R % FN;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            b[kk][j], a[kk][i], acc[i][j], 0, 0, 0, (int)sb, 0, (int)sa[i]);
        slot_dma(q);
        if constexpr (kk == 0)
          static_for_range<R * NL / NM, (R + 1) * NL / NM>([&](auto x) {
            constexpr int X = decltype(x)::value;
            if constexpr (X < FN) b[1][X] = b_frag(X, 1);
            else a[1][X - FN] = a_frag(X - FN, 1);
          });
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
      const float fb = sb_f32 ? __builtin_bit_cast(float, sb_raw) : e8m0_value(sb_raw);
      float f[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i)
        f[i] = (sa_f32 ? __builtin_bit_cast(float, sa[i]) : e8m0_value(sa[i])) * fb;
      i32x8_t a[2], b[2][FN];  // one row fragment of A at a time
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
        for (int j = 0; j < FN; ++j) b[kk][j] = b_frag(j, kk);
        a[kk] = a_frag(0, kk);
      }
      f32x16_t p[2];
      auto add_half = [&](auto tt, auto half) {  // half of sub-tile t's scaled sums
        constexpr int t = decltype(tt)::value, h = decltype(half)::value;
#pragma unroll
        for (int e = 8 * h; e < 8 * h + 8; ++e)
          acc[t / FN][t % FN][e] = __builtin_fmaf(f[t / FN], p[t & 1][e], acc[t / FN][t % FN][e]);
      };
      static_for<NS>([&](auto q) {
        constexpr int Q = decltype(q)::value, t = Q / 2, kk = Q % 2, i = t / FN, j = t % FN;
        f32x16_t& s = p[t & 1];
        if constexpr (kk == 0) s = f32x16_t{};
        s = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[kk][j], a[kk], s, 0, 0, 0, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (i + 1 < FM && j == FN - 1) a[kk] = a_frag(i + 1, kk);
        slot_dma(q);
        if constexpr (t > 0)
          add_half(std::integral_constant<int, t - 1>{}, std::integral_constant<int, kk>{});
        __builtin_amdgcn_sched_barrier(0);
      });
      add_half(std::integral_constant<int, FM * FN - 1>{}, std::integral_constant<int, 0>{});
      add_half(std::integral_constant<int, FM * FN - 1>{}, std::integral_constant<int, 1>{});
    }
  }

  // ---- Read-ahead (RING): while a stage is multiplied, the operands of the
  // next one are read from LDS into a second set of registers, so that no
  // matrix instruction waits for LDS at a stage's start.  The next stage then
  // has to have landed one step earlier, which takes a third buffer, and the
  // second set fits only beside the accumulators of the smaller tiles.
  struct Frags {
    i32x8_t a[2][FM], b[2][FN];
    uint32_t sa[FM], sb;
  };
  static constexpr int NL = 2 * (FM + FN);  // operand loads of a stage
  struct Ptrs {
    RowPtrs a;
    typename std::conditional<TB, RowPtrs, ColPtrs>::type b;
    const lds_t* s;
  };
  __device__ static __forceinline__ Ptrs ptrs(const lds_t* base, uint32_t wm, uint32_t wn) {
    Ptrs r;
    r.a = row_ptrs(base, wm * TM);
    if constexpr (TB)
      r.b = row_ptrs(base + A_BYTES, wn * TN);
    else
      r.b = col_ptrs(base + A_BYTES, wn);
    r.s = base + A_BYTES + B_BYTES;
    return r;
  }
  __device__ static __forceinline__ void load_scales(Frags& f, const Ptrs& r, uint32_t wm, uint32_t wn) {
    const uint32_t l32 = threadIdx.x & 31u;
#pragma unroll
    for (int i = 0; i < FM; ++i) f.sa[i] = *(const lds_u32_t*)(r.s + (wm * TM + i * 32 + l32) * 4);
    f.sb = *(const lds_u32_t*)(r.s + SA_BYTES + (wn * TN / kScaleBlock) * 4);
  }
  template <int X>
  __device__ static __forceinline__ void load_frag(Frags& f, const Ptrs& r) {
    constexpr int kk = X / (FM + FN), x = X % (FM + FN);
    if constexpr (x < FN) {
      if constexpr (TB) f.b[kk][x] = rows_frag(r.b, x, kk);
      else f.b[kk][x] = cols_frag(r.b, x, kk);
    } else {
      f.a[kk][x - FN] = rows_frag(r.a, x - FN, kk);
    }
  }

  __device__ static __forceinline__ void step_ring(f32x16_t (&acc)[FM][FN], const Frags& f, Frags& n,
                                                   const Ptrs& np, uint32_t wm, uint32_t wn,
                                                   bool sa_f32, bool sb_f32, const Src& c,
                                                   const Lanes& ln, const Stage& next) {
    constexpr int NS = 2 * FM * FN;
    auto behind = [&](auto q) {  // what rides behind slot q's matrix instruction
      constexpr int Q = decltype(q)::value;
      if constexpr (Q == 0) load_scales(n, np, wm, wn);
      static_for_range<Q * NL / NS, (Q + 1) * NL / NS>(
          [&](auto x) { load_frag<decltype(x)::value>(n, np); });
      static_for_range<Q * ND / NS, (Q + 1) * ND / NS>(
          [&](auto x) { dma_one<decltype(x)::value>(c, ln, next); });
    };
    if constexpr (HW) {
      static_for<NS>([&](auto q) {
        constexpr int Q = decltype(q)::value, kk = Q / (FM * FN), R = Q % (FM * FN);
        constexpr int i = R / FN, j = R % FN;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            f.b[kk][j], f.a[kk][i], acc[i][j], 0, 0, 0, (int)f.sb, 0, (int)f.sa[i]);
        __builtin_amdgcn_sched_barrier(0);
        behind(q);
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
      const float fb = sb_f32 ? __builtin_bit_cast(float, f.sb) : e8m0_value(f.sb);
      float s[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const uint32_t w = f.sa[i];
        s[i] = (sa_f32 ? __builtin_bit_cast(float, w) : e8m0_value(w)) * fb;
      }
      f32x16_t p[2];
      auto add_half = [&](auto tt, auto half) {
        constexpr int t = decltype(tt)::value, h = decltype(half)::value;
#pragma unroll
        for (int e = 8 * h; e < 8 * h + 8; ++e)
          acc[t / FN][t % FN][e] = __builtin_fmaf(s[t / FN], p[t & 1][e], acc[t / FN][t % FN][e]);
      };
      static_for<NS>([&](auto q) {
        constexpr int Q = decltype(q)::value, t = Q / 2, kk = Q % 2, i = t / FN, j = t % FN;
        f32x16_t& d = p[t & 1];
        if constexpr (kk == 0) d = f32x16_t{};
        if constexpr (MODE == MODE_EXACT) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_codes(f.b[kk][j], u),
                                                        widen_codes(f.a[kk][i], u), d, 0, 0, 0);
        } else {
          d = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.b[kk][j], f.a[kk][i], d, 0, 0, 0, 0,
                                                              0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        behind(q);
        if constexpr (t > 0)
          add_half(std::integral_constant<int, t - 1>{}, std::integral_constant<int, kk>{});
        __builtin_amdgcn_sched_barrier(0);
      });
      add_half(std::integral_constant<int, FM * FN - 1>{}, std::integral_constant<int, 0>{});
      add_half(std::integral_constant<int, FM * FN - 1>{}, std::integral_constant<int, 1>{});
    }
  }

  // The K loop with read-ahead.  Steps run in pairs (one per register set); a
  // stage past the last holds zeros and adds nothing.
  __device__ static __forceinline__ void loop_ring(f32x16_t (&acc)[FM][FN], uint32_t kt0,
                                                   uint32_t nk, uint32_t K, uint32_t wm, uint32_t wn,
                                                   bool sa_f32, bool sb_f32, const Src& c,
                                                   const Lanes& ln) {
    // stage 0 landed, the STAGES - 2 behind it in flight
    wait_vm<(STAGES - 2) * LPS>();
    barrier_lds();
    const uint32_t part = (K & 15u) ? nk - 1 : 0xffffffffu;  // the stage to clear the tail of
    if (kt0 == part) clear_tail(lds(), K & 127u);
    Frags f[2];
    {
      const Ptrs p0 = ptrs(lds(), wm, wn);
      load_scales(f[0], p0, wm, wn);
      static_for<NL>([&](auto x) { load_frag<decltype(x)::value>(f[0], p0); });
    }
    uint32_t cur = 0;  // buffer of stage kt
    auto step = [&](uint32_t kt, const Frags& now, Frags& then) {
      // stage kt + 1 landed; every wave has read stage kt and is done with kt - 1
      wait_vm<(STAGES - 3) * LPS>();
      barrier_lds();
      const uint32_t nb = cur + 1 == STAGES ? 0 : cur + 1;     // stage kt + 1
      const uint32_t pb = cur == 0 ? STAGES - 1 : cur - 1;     // stage kt - 1, free
      const Stage next = stage(c, ln, kt + STAGES - 1, pb);
      dma_scales(c, ln, next, kt + STAGES - 1);
      if (kt + 1 == part) clear_tail(lds() + nb * STAGE_BYTES, K & 127u);
      const Ptrs np = ptrs(lds() + nb * STAGE_BYTES, wm, wn);
      step_ring(acc, now, then, np, wm, wn, sa_f32, sb_f32, c, ln, next);
      cur = nb;
    };
    for (uint32_t kt = kt0; kt < c.kt1; kt += 2) {
      step(kt, f[0], f[1]);
      step(kt + 1, f[1], f[0]);
    }
  }

  // The K loop of a wave none of whose rows or columns is inside the matrix: it
  // loads its share, passes the same barriers as the others, and leaves the
  // matrix unit to the waves beside it (a group's last tile is seldom full).
  __device__ static __forceinline__ void loop_idle(uint32_t kt0, uint32_t nk, uint32_t K,
                                                   const Src& c, const Lanes& ln) {
    const uint32_t part = (K & 15u) ? nk - 1 : 0xffffffffu;
    uint32_t cur = 0;
    if constexpr (RING) {
      if (kt0 >= c.kt1) return;
      wait_vm<(STAGES - 2) * LPS>();
      barrier_lds();
      if (kt0 == part) clear_tail(lds(), K & 127u);
    }
    const uint32_t end = RING ? kt0 + (c.kt1 - kt0 + 1) / 2 * 2 : c.kt1;
    for (uint32_t kt = kt0; kt < end; ++kt) {
      wait_vm<(STAGES - (RING ? 3 : 2)) * LPS>();
      barrier_lds();
      const uint32_t nb = cur + 1 == STAGES ? 0 : cur + 1;
      const Stage next = stage(c, ln, kt + STAGES - 1, cur == 0 ? STAGES - 1 : cur - 1);
      dma_scales(c, ln, next, kt + STAGES - 1);
      static_for<ND>([&](auto x) { dma_one<decltype(x)::value>(c, ln, next); });
      if (RING && kt + 1 == part) clear_tail(lds() + nb * STAGE_BYTES, K & 127u);
      if (!RING && kt == part) clear_tail(lds() + cur * STAGE_BYTES, K & 127u);
      cur = nb;
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
      const uint32_t full = __builtin_amdgcn_readfirstlane(groups.first_task[a.G]);
      const uint32_t tails = __builtin_amdgcn_readfirstlane(groups.first_tail[a.G]);
      const uint32_t large = tails & 0xffffu;
      if (blockIdx.x >= full + (large + (tails >> 16)) * loops_n) return;  // the whole workgroup
      if (blockIdx.x < full) {
        const uint32_t u = logical_wg(a.remap, full);
        g = find_group(groups.first_task, a.G, u);
        t = block_coord((groups.first_row[g + 1] - groups.first_row[g]) / BM, loops_n, a.off, a.dir,
                        u - groups.first_task[g]);
        t.m = __builtin_amdgcn_readfirstlane(t.m);
        t.n = __builtin_amdgcn_readfirstlane(t.n);
      } else {
        const uint32_t v = blockIdx.x - full;
        const uint32_t r = v / loops_n;
        g = r < large ? find_group<0, 0xffffu>(groups.first_tail, a.G, r)
                      : find_group<16, 0xffffu>(groups.first_tail, a.G, r - large);
        t.m = __builtin_amdgcn_readfirstlane((groups.first_row[g + 1] - groups.first_row[g]) / BM);
        t.n = v % loops_n;
      }
      row0 = __builtin_amdgcn_readfirstlane(groups.first_row[g]);
      rows = __builtin_amdgcn_readfirstlane(groups.first_row[g + 1]) - row0;
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
    c.ldb = a.ldb;
    c.K = a.K;
    c.kt1 = kt1;
    c.wave = wave;
    // the scales this wave loads: A's rows, or the tile's blocks of columns
    const bool sa_f32 = !HW && a.sa_f32, sb_f32 = !HW && a.sb_f32;
    const bool for_a = wave < (uint32_t)SA_N;
    c.s_f32 = for_a ? sa_f32 : sb_f32;
    const int64_t ss = c.s_f32 ? 4 : 1;
    const uint32_t nb = n0 / kScaleBlock, nbs = (a.N + kScaleBlock - 1) / kScaleBlock - nb;
    if (for_a) {
      c.s = a.sa + arow * a.ldsa * ss;
      c.s_step = ss;
    } else {
      c.s = a.sb + ((int64_t)g * a.strideSB + (int64_t)nb * (TB ? a.ldsb : 1)) * ss;
      c.s_step = (TB ? 1 : a.ldsb) * ss;
    }
    c.lda32 = (uint32_t)a.lda;
    c.ldb32 = (uint32_t)a.ldb;
    const Tile tile{c.lda32, c.ldb32, a.K, rows_left, cols_left,
                    (uint32_t)((for_a ? a.ldsa : TB ? a.ldsb : 1) * ss), nbs};
    const Lanes ln = lanes(tile, wave, lane);

    f32x16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    // ---- K loop: at the top of a step stage kt must have landed and the
    // STAGES - 2 stages behind it may still be in flight
    for (uint32_t s = 0; s < (uint32_t)STAGES - 1; ++s) {
      const Stage st = stage(c, ln, kt0 + s, s);
      dma_scales(c, ln, st, kt0 + s);
      static_for<ND>([&](auto x) { dma_one<decltype(x)::value>(c, ln, st); });
    }
    if (wm * TM >= rows_left || wn * TN >= cols_left) {
      loop_idle(kt0, a.nk, a.K, c, ln);
    } else if constexpr (RING) {
      if (kt0 < kt1) loop_ring(acc, kt0, a.nk, a.K, wm, wn, sa_f32, sb_f32, c, ln);
    } else {
      uint32_t buf = 0;
      for (uint32_t kt = kt0; kt < kt1; ++kt) {
        wait_vm<(STAGES - 2) * LPS>();
        barrier_lds();
        const uint32_t nb = buf == 0 ? STAGES - 1 : buf - 1;  // the buffer read in the last step
        const Stage next = stage(c, ln, kt + STAGES - 1, nb);
        dma_scales(c, ln, next, kt + STAGES - 1);
        lds_t* base = lds() + buf * STAGE_BYTES;
        if (kt + 1 == a.nk && (a.K & 15u)) clear_tail(base, a.K & 127u);
        compute(acc, base, wm, wn, sa_f32, sb_f32, c, ln, next);
        buf = buf + 1 == STAGES ? 0 : buf + 1;
      }
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
    using S = Strips<FM, FN>;
    lds_t* const strips = lds() + wave * S::BYTES;
    if (!GROUPED && a.part != nullptr)
      S::template store<false>(strips, acc, wm * TM, wn * TN, o);
    else
      S::template store<true>(strips, acc, wm * TM, wn * TN, o);
  }
};

template <int BM, int BN, int WM, int WN, int STAGES, bool TB, int MODE, bool GROUPED>
__global__ void __launch_bounds__(64 * WM * WN) block_gemm_kernel(BlockGemmArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  BlockGemm<BM, BN, WM, WN, STAGES, TB, MODE, GROUPED>::run(a);
#endif
}

}  // namespace bst
