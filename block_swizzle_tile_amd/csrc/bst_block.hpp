// bst_block.hpp -- what the block-scaled 8-bit operators share on the device:
// scale decoding, group tables, the masked row stores of an output tile, and
// the fixed-order sum of split partials.
#pragma once

#include "bst.h"
#include "bst_block.h"
#include "bst_kernel_dma.hpp"

namespace bst {

// Defined with the C ABI's other host code: records the message that
// bst_last_error() returns on this thread, and passes the status through.
bst_status set_error(bst_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int device_cu_count();

constexpr uint32_t kScaleBlock = 128;  // values that share a scale

// 2^(e - 127); byte 0 is the subnormal 2^-127, byte 255 NaN.
__device__ __forceinline__ float e8m0_value(uint32_t e) {
  const uint32_t bits = e == 0u ? 0x00400000u : e == 255u ? 0x7fc00000u : e << 23;
  return __builtin_bit_cast(float, bits);
}

// Groups of stacked rows, in LDS: each group's first row, its first task among
// the full tile-rows, and its first tile-row among the partial ones (a group
// has at most one; those of more than half a tile's rows are counted in the low
// 16 bits, the others in the high ones), with the totals behind the last group.
// Partial tiles come after all full ones, and the smaller ones last: they are
// the shorter tasks, and workgroups start in order, so the chip's last round
// is filled with them.
struct RowGroups {
  uint32_t first_row[kMaxGroups + 1];
  uint32_t first_task[kMaxGroups + 1];
  uint32_t first_tail[kMaxGroups + 1];
};

// Built by wave 0 with a scan over the groups (lane l holds groups l*per ..):
// sizes below 0 count as 0, and a running sum past total_m is cut to it.
// bm, loops_n: rows per tile-row and tasks per tile-row.
__device__ inline void build_row_groups(RowGroups& t, const int32_t* group_m, uint32_t G,
                                        uint32_t total_m, uint32_t bm, uint32_t loops_n) {
  if (threadIdx.x < 64u) {
    const uint32_t lane = threadIdx.x, per = (G + 63u) / 64u;
    const uint32_t g0 = lane * per < G ? lane * per : G, g1 = g0 + per < G ? g0 + per : G;
    int64_t rows = 0;
    for (uint32_t g = g0; g < g1; ++g) rows += group_m[g] > 0 ? group_m[g] : 0;
    int64_t sum = rows;
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up((long long)sum, d);
      if ((int)lane >= d) sum += o;
    }
    int64_t at = sum - rows;  // rows before this lane's groups, not yet cut
    uint32_t tasks = 0, tails = 0;
    for (uint32_t g = g0; g < g1; ++g) {
      const uint32_t lo = at < (int64_t)total_m ? (uint32_t)at : total_m;
      at += group_m[g] > 0 ? group_m[g] : 0;
      const uint32_t hi = at < (int64_t)total_m ? (uint32_t)at : total_m;
      t.first_row[g] = lo;
      t.first_task[g] = tasks;
      t.first_tail[g] = tails;
      tasks += (hi - lo) / bm * loops_n;
      const uint32_t rest = (hi - lo) % bm;
      tails += rest > bm / 2 ? 1u : rest != 0 ? 0x10000u : 0u;
      if (g + 1 == G) t.first_row[G] = hi;
    }
    uint32_t ts = tasks, ls = tails;
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = (uint32_t)__shfl_up((int)ts, d), l = (uint32_t)__shfl_up((int)ls, d);
      if ((int)lane >= d) {
        ts += o;
        ls += l;
      }
    }
    for (uint32_t g = g0; g < g1; ++g) {
      t.first_task[g] += ts - tasks;
      t.first_tail[g] += ls - tails;
    }
    if (lane == 63u) {
      t.first_task[G] = ts;
      t.first_tail[G] = ls;
    }
  }
  __syncthreads();
}

// The last group whose first entry is at most x (groups without entries of
// their own share the next one's).
template <int SHIFT = 0, uint32_t MASK = 0xffffffffu>
__device__ __forceinline__ uint32_t find_group(const uint32_t* first, uint32_t G, uint32_t x) {
  uint32_t lo = 0, hi = G - 1;
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) >> 1;
    if ((first[mid] >> SHIFT & MASK) <= x) lo = mid; else hi = mid - 1;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// ------------------------------------------------------------ output ------
__device__ __forceinline__ uint32_t pack2(float a, float b, uint32_t kind) {
  if (kind == OUT_BF16) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    b2 v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, v);
  }
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  h2 v;
  v[0] = (_Float16)a;
  v[1] = (_Float16)b;
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float out_value(const uint8_t* p, uint32_t kind) {
  if (kind == OUT_F32) return *(const float*)p;
  if (kind == OUT_BF16) return __builtin_bit_cast(float, (uint32_t)(*(const uint16_t*)p) << 16);
  return (float)*(const _Float16*)p;
}

__device__ __forceinline__ void put_value(uint8_t* p, float v, uint32_t kind) {
  if (kind == OUT_F32)
    *(float*)p = v;
  else
    *(uint16_t*)p = (uint16_t)pack2(v, 0.0f, kind);
}

// N consecutive outputs (N = 4 or 8): with `add` the addend joins in fp32
// before the one rounding.  whole: all N are inside the row and both rows are
// aligned for vector access; otherwise `live` of them go one by one.
template <int N>
__device__ __forceinline__ void put_run(uint8_t* dst, const uint8_t* add, float (&v)[N],
                                        uint32_t live, bool whole, uint32_t kind) {
  const uint32_t es = kind == OUT_F32 ? 4u : 2u;
  if (whole) {
    if (kind == OUT_F32) {
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
        f32x4_t o = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        if (add != nullptr) o += ((const f32x4_t*)add)[q];
        ((f32x4_t*)dst)[q] = o;
      }
    } else {
      uint32_t a[N / 2], o[N / 2];
      if (add != nullptr) {
        if constexpr (N == 8) {
          const u32x4_t w = *(const u32x4_t*)add;
          a[0] = w[0]; a[1] = w[1]; a[2] = w[2]; a[3] = w[3];
        } else {
          const u32x2_t w = *(const u32x2_t*)add;
          a[0] = w[0]; a[1] = w[1];
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const uint16_t h = (uint16_t)(a[e / 2] >> (16 * (e & 1)));
          v[e] += out_value((const uint8_t*)&h, kind);
        }
      }
#pragma unroll
      for (int e = 0; e < N / 2; ++e) o[e] = pack2(v[2 * e], v[2 * e + 1], kind);
      if constexpr (N == 8)
        *(u32x4_t*)dst = u32x4_t{o[0], o[1], o[2], o[3]};
      else
        *(u32x2_t*)dst = u32x2_t{o[0], o[1]};
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if ((uint32_t)e < live)
      put_value(dst + e * es, v[e] + (add != nullptr ? out_value(add + e * es, kind) : 0.0f), kind);
}

// Where a tile goes: the final matrix, or a slice's partial sums (fp32, rows
// of `ld` elements).
struct OutTile {
  uint8_t* dst;        // the tile's first element
  const uint8_t* add;  // the addend's, or null
  int64_t ld_bytes, ldadd_bytes;
  uint32_t rows, cols;  // valid rows and columns of the tile
  uint32_t kind;
  bool vec;  // rows of dst (and add) start on 16-byte boundaries
};

// Stores a wave's TM x TN sub-tile held as 32x32 accumulators (lane l: row
// l & 31 of the fragment, columns 8q + 4(l >> 5) + 0..3), one strip of 32 rows
// at a time through the wave's own LDS, so that global stores are runs of a
// row.  Waves do not wait for each other: LDS accesses of one wave complete in
// order.  Whole rows of vectors have two forms of their own, because nothing
// hides a tile's epilogue: 16-bit outputs are packed before they go through
// LDS, 32-bit ones are not.  One unrolled form for all was slower by its own
// code and waits (one 256x256 tile per workgroup, 16 of them, K = 128: 9.6 us
// against 6.7; 8192 rows over 8 groups of 4096 x 2048: 95 against 91), and so
// were 16-bit strips of 128 rows (92).
//
// THROUGH: whole runs go through the L2 to memory, so that they do not stay
// dirty in it, take the place of operand panels and wait for the write-back at
// the kernel's end: 8192 rows over 8 groups of 4096 x 2048 99.9 -> 95.5 us,
// 8192 x 8192 x 4096 272 -> 265, 1024 x 2048 x 4096 19.7 -> 19.4.  Not for what
// the next launch reads or what was read into the L2 just before (partial
// sums; a gradient with an addend: 265 -> 278 us at 8192 x 4096 x 4096).  It
// needs a tile whose rows span less than 2 GiB.
template <int FM, int FN>
struct Strips {
  static constexpr int TN = FN * 32;
  // 32-bit strips: rows are padded by 4 floats, so that the 32 rows' quads fall
  // on different banks
  static constexpr int PITCH = TN + 4;
  static constexpr int BYTES = 32 * PITCH * 4;
  static constexpr int CPR = TN / 8;    // runs of 8 columns per row
  static constexpr int RPI = 64 / CPR;  // rows one pass of the wave stores
  typedef __attribute__((address_space(3))) f32x4_t lds_f4_t;

  // 16-bit rows of TN * 2 bytes; their 16-byte chunks are XORed by the row, so
  // that 8 rows' chunks (write) and a row's chunks (read) fall on different banks
  static __device__ __forceinline__ uint32_t at16(uint32_t row, uint32_t ch) {
    return row * (TN * 2) + ((ch ^ (CPR == 8 ? row & 7u : (row >> 1) & 3u)) << 4);
  }
  template <uint32_t KIND>
  static __device__ __forceinline__ void strip16(lds_t* s, const f32x16_t (&acc)[FN]) {
    const uint32_t lane = threadIdx.x & 63u, r = lane & 31u, hi = lane >> 5;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        // quads q and q + 1 of a row are in lanes l and l + 32: after the swaps
        // lane l holds all 8 columns of q, and l + 32 those of q + 1
        u32x2_t v[2];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const uint32_t x = pack2(acc[j][4 * q + 2 * d], acc[j][4 * q + 2 * d + 1], KIND);
          const uint32_t y = pack2(acc[j][4 * q + 4 + 2 * d], acc[j][4 * q + 5 + 2 * d], KIND);
          const auto w = __builtin_amdgcn_permlane32_swap(x, y, false, false);
          v[d] = u32x2_t{w[0], w[1]};
        }
        *(lds_u32x4_t*)(s + at16(r, j * 4 + q + hi)) = u32x4_t{v[0][0], v[1][0], v[0][1], v[1][1]};
      }
  }
  static __device__ __forceinline__ void strip32(lds_t* s, const f32x16_t (&acc)[FN]) {
    const uint32_t lane = threadIdx.x & 63u, r = lane & 31u, hi = lane >> 5;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(lds_f4_t*)(s + (r * PITCH + j * 32 + 8 * q + 4 * hi) * 4) =
            f32x4_t{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
  }
  static __device__ __forceinline__ void written() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

  template <bool THROUGH>
  static __device__ __forceinline__ void store(lds_t* s, f32x16_t (&acc)[FM][FN], uint32_t m0,
                                               uint32_t n0, const OutTile& o) {
    if (m0 >= o.rows || n0 >= o.cols) return;  // wave-uniform, as all branches but the last
    const uint32_t lane = threadIdx.x & 63u, row = lane / CPR, c = (lane % CPR) * 8;
    const uint32_t n = n0 + c;
    const bool runs = o.vec && o.cols % 8 == 0;
    const __amdgpu_buffer_rsrc_t through =
        __builtin_amdgcn_make_buffer_rsrc(o.dst, (short)0, (int)0x7fffffff, 0x00020000);
    auto put = [&](uint32_t m, uint32_t off, u32x4_t v) {  // 16 bytes, off bytes into row m
      if constexpr (THROUGH)
        __builtin_amdgcn_raw_buffer_store_b128(v, through, m * (uint32_t)o.ld_bytes + off, 0, 16);
      else
        *(u32x4_t*)(o.dst + (int64_t)m * o.ld_bytes + off) = v;
    };
    if (runs && o.kind != OUT_F32 && o.add == nullptr) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if (o.kind == OUT_BF16) strip16<OUT_BF16>(s, acc[i]);
        else strip16<OUT_F16>(s, acc[i]);
        written();
#pragma unroll
        for (int p = 0; p < 32 / RPI; ++p) {
          const uint32_t r = p * RPI + row, m = m0 + i * 32 + r;
          const u32x4_t v = *(const lds_u32x4_t*)(s + at16(r, lane % CPR));
          if (m < o.rows && n < o.cols) put(m, n * 2, v);
        }
        written();
      }
    } else if (runs && o.kind == OUT_F32) {
      constexpr int P = 32 / RPI;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        strip32(s, acc[i]);
        written();
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const uint32_t r = p * RPI + row, m = m0 + i * 32 + r;
          f32x4_t x = *(const lds_f4_t*)(s + (r * PITCH + c) * 4);
          f32x4_t y = *(const lds_f4_t*)(s + (r * PITCH + c + 4) * 4);
          if (m < o.rows && n < o.cols) {
            if (o.add != nullptr) {
              const f32x4_t* a = (const f32x4_t*)(o.add + (int64_t)m * o.ldadd_bytes + n * 4);
              x += a[0];
              y += a[1];
            }
            put(m, n * 4, __builtin_bit_cast(u32x4_t, x));
            put(m, n * 4 + 16, __builtin_bit_cast(u32x4_t, y));
          }
        }
        written();
      }
    } else {
      const uint32_t es = o.kind == OUT_F32 ? 4u : 2u;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        strip32(s, acc[i]);
        written();
#pragma unroll 1
        for (uint32_t r = row; r < 32; r += RPI) {
          const uint32_t m = m0 + i * 32 + r;
          const f32x4_t x = *(const lds_f4_t*)(s + (r * PITCH + c) * 4);
          const f32x4_t y = *(const lds_f4_t*)(s + (r * PITCH + c + 4) * 4);
          float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
          if (m < o.rows && n < o.cols) {
            uint8_t* d = o.dst + (int64_t)m * o.ld_bytes + (int64_t)n * es;
            const uint8_t* ad = o.add ? o.add + (int64_t)m * o.ldadd_bytes + (int64_t)n * es : nullptr;
            put_run<8>(d, ad, v, o.cols - n, o.vec && o.cols - n >= 8u, o.kind);
          }
        }
        written();
      }
    }
  }
};

// Sum of the split partials in slice order, the addend, and the one rounding.
// part: [split][count][rows][pitch] fp32, pitch a multiple of 4.
struct ReduceArgs {
  const float* part;
  uint8_t* dst;
  const uint8_t* add;
  int64_t ld, stride, ldadd, strideadd;  // elements
  uint32_t split, rows, cols, pitch;
  uint32_t kind, vec;
  FastDiv quads, by_rows;  // pitch / 4, rows
  uint32_t total;          // count * rows * pitch / 4
};

static __global__ void __launch_bounds__(256) sum_partials(ReduceArgs a) {
  const uint32_t es = a.kind == OUT_F32 ? 4u : 2u;
  const int64_t slice = (int64_t)a.total * 4;
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < a.total; i += gridDim.x * 256u) {
    const uint32_t rr = a.quads.div(i), q = i - rr * a.quads.d;
    const uint32_t g = a.by_rows.div(rr), r = rr - g * a.rows;
    const float* p = a.part + (int64_t)i * 4;
    // in slice order, eight slices in flight
    f32x4_t s = *(const f32x4_t*)p;
    uint32_t k = 1;
    for (; k + 8 <= a.split; k += 8) {
      f32x4_t v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = *(const f32x4_t*)(p + (k + u) * slice);
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    f32x4_t v[7];
#pragma unroll
    for (int u = 0; u < 7; ++u)
      if (k + u < a.split) v[u] = *(const f32x4_t*)(p + (k + u) * slice);
#pragma unroll
    for (int u = 0; u < 7; ++u)
      if (k + u < a.split) s += v[u];
    const uint32_t n = q * 4;
    if (n >= a.cols) continue;
    float w[4] = {s[0], s[1], s[2], s[3]};
    uint8_t* d = a.dst + (g * a.stride + r * a.ld + n) * es;
    const uint8_t* ad = a.add ? a.add + (g * a.strideadd + r * a.ldadd + n) * es : nullptr;
    put_run<4>(d, ad, w, a.cols - n, a.vec && a.cols - n >= 4u, a.kind);
  }
}

}  // namespace bst
