// bst_moe.hpp -- the kernels around a mixture of experts: a stable counting
// sort of the router's choices, the copy of tokens to their experts' rows, the
// weighted sum back, and its gradient.
//
// All but the sort move whole rows and are bound by memory: every token and
// every row is read or written once, token by token, so that a token's k copies
// (or addends) meet in one thread's registers.
#pragma once

#include "bst_values.hpp"

namespace bst {

// ---------------------------------------------------------------- sort ----
struct MoeSortArgs {
  const void* expert;
  int32_t* row_of;
  int32_t* group_m;
  uint32_t* counts;  // [chunks][pitch]: rows of each expert in each chunk
  int64_t first;
  uint32_t n, G, pitch, chunk, chunks;
};

// The expert's index here, or G where it is not here.  (A 64-bit id less `first` may
// leave 64 bits: compared before it is subtracted.)
template <typename Id>
__device__ __forceinline__ uint32_t expert_key(const MoeSortArgs& a, Id id) {
  const int64_t e = id;
  return e >= a.first && e - a.first < (int64_t)a.G ? (uint32_t)(e - a.first) : a.G;
}

// E = 16 / sizeof(Id) consecutive choices, and `none` for those past n.
template <typename Id, int E>
__device__ __forceinline__ void expert_run(const MoeSortArgs& a, uint32_t i, Id none, Id (&id)[E]) {
  typedef Id run_t __attribute__((ext_vector_type(E), aligned(sizeof(Id))));
  if (i + E <= a.n) {
    const run_t v = *(const run_t*)((const Id*)a.expert + i);
#pragma unroll
    for (int e = 0; e < E; ++e) id[e] = v[e];
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) id[e] = i + e < a.n ? ((const Id*)a.expert)[i + e] : none;
  }
}

// One launch: workgroup g finds expert g's rows by itself.  Each wave has a
// stretch of the choices and counts those of g and of the experts before g; with
// all waves' counts it knows its first row, and goes through its stretch again,
// where the bits of a ballot are a lane's place.  Every workgroup reads all
// choices, from the L2.
template <typename Id, int NW>
__global__ void __launch_bounds__(64 * NW) moe_sort_one(MoeSortArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef typename std::make_unsigned<Id>::type U;
  constexpr int E = 16 / (int)sizeof(Id);
  constexpr uint32_t STEP = 64u * E;
  __shared__ uint32_t eq_of[NW], less_of[NW];
  const uint32_t g = blockIdx.x, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
  const uint32_t stretch = ((a.n + NW - 1) / NW + STEP - 1) / STEP * STEP;
  const uint32_t i0 = min(wave * stretch, a.n), i1 = min(i0 + stretch, a.n);
  // an id less the first expert, as an unsigned number, is below G if it is here, and
  // below g if it comes before g
  const U first = (U)a.first;
  const Id mine = (Id)(first + g), none = (Id)(first + (U)a.G);
  uint32_t eq = 0, less = 0;
  Id id[E];
#pragma unroll 4
  for (uint32_t i = i0; i < i1; i += STEP) {
    expert_run<Id, E>(a, i + lane * E, none, id);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      eq += (uint32_t)__popcll(__ballot(id[e] == mine));
      less += (uint32_t)__popcll(__ballot((U)id[e] - first < (U)g));
    }
  }
  if (lane == 0) {
    eq_of[wave] = eq;
    less_of[wave] = less;
  }
  __syncthreads();
  uint32_t row = 0, total = 0;
#pragma unroll
  for (uint32_t w = 0; w < (uint32_t)NW; ++w) {
    row += less_of[w] + (w < wave ? eq_of[w] : 0u);
    total += eq_of[w];
  }
  if (threadIdx.x == 0) a.group_m[g] = (int32_t)total;
  if (eq != 0) {
    for (uint32_t i = i0; i < i1; i += STEP) {
      expert_run<Id, E>(a, i + lane * E, none, id);
      uint64_t m[E];
      uint32_t at = row;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        m[e] = __ballot(id[e] == mine);
        at = __builtin_amdgcn_mbcnt_hi((uint32_t)(m[e] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m[e], at));
        row += (uint32_t)__popcll(m[e]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (id[e] == mine) a.row_of[i + lane * E + e] = (int32_t)at++;
    }
  }
  // choices without a row: the workgroups share them out
  for (uint32_t i = i0 + g * STEP; i < i1; i += gridDim.x * STEP) {
    expert_run<Id, E>(a, i + lane * E, mine, id);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((U)id[e] - first >= (U)a.G && i + lane * E + e < a.n) a.row_of[i + lane * E + e] = -1;
  }
#endif
}

// Four choices' keys, STRIDE apart from i on, those past `end` as G.
template <typename Id, int STRIDE>
__device__ __forceinline__ void four_keys(const MoeSortArgs& a, uint32_t i, uint32_t end, uint32_t (&key)[4]) {
  Id id[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) id[u] = ((const Id*)a.expert)[min(i + u * STRIDE, end - 1)];
#pragma unroll
  for (int u = 0; u < 4; ++u) key[u] = i + u * STRIDE < end ? expert_key<Id>(a, id[u]) : a.G;
}

// Two launches for many: chunks of choices are counted, then every chunk's
// workgroup adds up the counts of all chunks for its experts' first rows and
// ranks its choices in order.
template <typename Id>
__global__ void __launch_bounds__(256) moe_count(MoeSortArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ uint32_t hist[kMaxGroups + 4];
  for (uint32_t g = threadIdx.x; g < a.pitch; g += 256u) hist[g] = 0;
  __syncthreads();
  const uint32_t i0 = blockIdx.x * a.chunk, i1 = min(i0 + a.chunk, a.n);
  for (uint32_t i = i0; i < i1; i += 1024u) {
    uint32_t key[4];
    four_keys<Id, 256>(a, i + threadIdx.x, i1, key);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (key[u] < a.G) atomicAdd(&hist[key[u]], 1u);  // whole numbers: any order gives the same
  }
  __syncthreads();
  for (uint32_t g = threadIdx.x; g < a.pitch; g += 256u) a.counts[(size_t)blockIdx.x * a.pitch + g] = hist[g];
#endif
}

template <typename Id>
__global__ void __launch_bounds__(256) moe_place(MoeSortArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ uint32_t all[1024], before[1024];   // [part][expert] sums, then the experts'
  __shared__ uint32_t next[4][kMaxGroups];       // each wave's next row of each expert
  __shared__ uint32_t wave_sum[4];
  const uint32_t tid = threadIdx.x, wave = tid >> 6, lane = tid & 63u;
  // ---- this wave's part of the chunk, the first 256 choices of it (for a sort of up
  // to 2^19 all of it) in registers
  const uint32_t share = a.chunk / 4;
  const uint32_t i0 = min(blockIdx.x * a.chunk + wave * share, a.n);
  const uint32_t i1 = min(i0 + share, a.n);
  uint32_t key[4] = {a.G, a.G, a.G, a.G};
  if (i0 < i1) four_keys<Id, 64>(a, i0 + lane, i1, key);
  // ---- counts over all chunks and over those before this one: the threads of
  // one expert quad share the chunks out
  const uint32_t quads = a.pitch / 4, parts = 256u / quads;
  {
    const uint32_t q = tid % quads, p = tid / quads;
    if (p < parts) {
      const uint32_t per = (a.chunks + parts - 1) / parts;
      const uint32_t c0 = min(p * per, a.chunks), c1 = min(c0 + per, a.chunks);
      u32x4_t t = {0u, 0u, 0u, 0u}, b = {0u, 0u, 0u, 0u};
      const uint32_t* src = a.counts + q * 4;
      uint32_t c = c0;
      for (; c + 8 <= c1; c += 8) {
        u32x4_t v[8];
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u) v[u] = *(const u32x4_t*)(src + (size_t)(c + u) * a.pitch);
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u) {
          t += v[u];
          if (c + u < blockIdx.x) b += v[u];
        }
      }
      for (; c < c1; ++c) {
        const u32x4_t v = *(const u32x4_t*)(src + (size_t)c * a.pitch);
        t += v;
        if (c < blockIdx.x) b += v;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        all[p * a.pitch + q * 4 + e] = t[e];
        before[p * a.pitch + q * 4 + e] = b[e];
      }
    }
  }
#pragma unroll
  for (uint32_t w = 0; w < 4; ++w)
    for (uint32_t g = tid; g < a.G; g += 256u) next[w][g] = 0;
  __syncthreads();
  // ---- thread's quad of experts: first rows by a scan over the experts
  uint32_t t[4] = {0, 0, 0, 0}, b[4] = {0, 0, 0, 0}, sum = 0;
  if (tid < quads)
    for (uint32_t p = 0; p < parts; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[e] += all[p * a.pitch + tid * 4 + e];
        b[e] += before[p * a.pitch + tid * 4 + e];
      }
#pragma unroll
  for (int e = 0; e < 4; ++e) sum += t[e];
  uint32_t scan = sum;
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)scan, d);
    if ((int)lane >= d) scan += o;
  }
  if (lane == 63u) wave_sum[wave] = scan;
  // ---- choices of each expert in each wave's part of the chunk
  for (uint32_t i = i0; i < i1; i += 256u) {
    if (i != i0) four_keys<Id, 64>(a, i + lane, i1, key);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (key[u] < a.G) atomicAdd(&next[wave][key[u]], 1u);
  }
  __syncthreads();
  if (tid < quads) {
    uint32_t row = scan - sum;
#pragma unroll
    for (uint32_t w = 0; w < 4; ++w)
      if (w < wave) row += wave_sum[w];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t g = tid * 4 + e;
      if (g < a.G) {
        if (blockIdx.x == 0) a.group_m[g] = (int32_t)t[e];
        uint32_t at = row + b[e];
#pragma unroll
        for (uint32_t w = 0; w < 4; ++w) {
          const uint32_t n = next[w][g];
          next[w][g] = at;
          at += n;
        }
      }
      row += t[e];
    }
  }
  __syncthreads();
  // ---- rows: a wave goes through its part 64 choices at a time.  Lanes of the
  // same expert find each other by the bits of its index; the lane's rank among
  // them is its place, and the last of them moves the expert's next row on.
  volatile uint32_t* const mine = next[wave];
  uint32_t bits = 0;
  while (bits < 11u && (a.G >> bits) != 0) ++bits;
  for (uint32_t i = i0; i < i1; i += 256u) {  // wave-uniform
    if (share > 256u) four_keys<Id, 64>(a, i + lane, i1, key);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t k = key[u], at = i + u * 64 + lane;
      uint64_t same = ~0ull;
      for (uint32_t d = 0; d < bits; ++d) {
        const uint64_t m = __ballot((k >> d) & 1u);
        same &= (k >> d) & 1u ? m : ~m;
      }
      const uint32_t rank = (uint32_t)__popcll(same & ((1ull << lane) - 1ull));
      uint32_t row = 0;
      if (k < a.G) row = mine[k];
      if (k < a.G && (same >> lane) == 1ull) mine[k] = row + rank + 1u;
      if (at < i1) a.row_of[at] = k < a.G ? (int32_t)(row + rank) : -1;
    }
  }
#endif
}

// ------------------------------------------------------------ row moves ----
// Large moves (is_far) store past the caches and load rows that are read once so: gather
// of 8192 x 8 rows of 2048 bf16 and their weighted sum 122 us without and 102 with it,
// 4096 x 8 rows 56.3 and 53.7, 2048 x 4 rows 19.4 and 17.5 (rows that the last-level
// cache has not seen of late; of those that it has, 4096 x 8 rows 131 us and 143 for
// both, the gradient and its sum, 8192 x 8 312 and 279).
struct MoeRows {  // a matrix whose rows are copied: bytes
  const uint8_t* x;
  uint8_t* r;
  int64_t ldx, ldr;
  uint32_t bytes;   // of a row
  uint32_t pieces;  // of 16 bytes, the last one perhaps shorter
  FastDiv by_pieces;
};

struct MoeGatherArgs {
  MoeRows m[2];  // the rows, and their scales (pieces = 0: none)
  const int32_t* row_of;
  uint32_t T, k, rows;
};

// One piece of a token to its k rows: 8192 x 8 rows of 2048 bf16, 302 MB, 51 us, 5.9
// TB/s; 16 x 4 rows of 4096 2.1 us, a launch and two loads in turn.  A last piece that is not whole starts
// earlier and writes the bytes that it shares with the piece before again.
template <bool FAR>
__device__ __forceinline__ void copy_piece(const MoeGatherArgs& a, const MoeRows& m, uint32_t i) {
  const uint32_t t = m.by_pieces.div(i), c = i - t * m.pieces;
  const int32_t* at = a.row_of + (int64_t)t * a.k;
  const uint8_t* x = m.x + (int64_t)t * m.ldx;
  if (m.bytes >= 16u) {
    const uint32_t off = min(c * 16u, m.bytes - 16u);
    const u32x4_t v = load16(x + off);
    for (uint32_t j0 = 0; j0 < a.k; j0 += 8) {  // eight rows' numbers are asked for together
      uint32_t row[8];
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u) row[u] = (uint32_t)at[min(j0 + u, a.k - 1)];
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u)
        if (j0 + u < a.k && row[u] < a.rows) store16<FAR>(m.r + (int64_t)row[u] * m.ldr + off, v);
    }
  } else {
    for (uint32_t j = 0; j < a.k; ++j) {
      const uint32_t row = (uint32_t)at[j];
      if (row >= a.rows) continue;
      for (uint32_t b = 0; b < m.bytes; ++b) m.r[(int64_t)row * m.ldr + b] = x[b];
    }
  }
}

template <bool FAR>
__global__ void __launch_bounds__(256) moe_gather_kernel(MoeGatherArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t n = a.T * a.m[0].pieces;  // both counts fit 32 bits (checked by the host)
  if (i < n)
    copy_piece<FAR>(a, a.m[0], i);
  else if (i - n < a.T * a.m[1].pieces)
    copy_piece<FAR>(a, a.m[1], i - n);
#endif
}

// -------------------------------------------------------- weighted sums ----
struct MoeCombineArgs {
  const uint8_t* R;
  const uint8_t* w;    // null: ones
  const uint8_t* add;  // null: none
  uint8_t* Y;
  const int32_t* row_of;
  int64_t ldr, ldadd, ldy;  // bytes
  uint32_t T, k, H, rows;
  uint32_t pieces;  // of a lane's values per row
  uint32_t wkind, ykind;
  FastDiv by_pieces;
};

__device__ __forceinline__ float weight(const uint8_t* w, int64_t i, uint32_t kind) {
  return w == nullptr ? 1.0f : out_value(w + i * (kind == X_F32 ? 4 : 2), kind);
}

// Columns of a lane: 16 bytes of a row, so that a wave's stores of fp32 are whole lines
// too.
template <int KIND>
constexpr int kCols = KIND == X_F32 ? 4 : 8;

// One thread, kCols columns of one token.  Rows are loaded four at a time without
// branches: a choice without a row reads row 0 and counts as zero.  (Eight at a time:
// 8191 x 8 rows of 2048 bf16 52.6 us, so 49.1.)  Bound by memory: those are 302 MB, 6.2
// TB/s; 16 x 4 rows of 4096, by three loads that wait for each other, 2.8 us.
template <int KIND, bool FAR>
__global__ void __launch_bounds__(256) moe_combine_kernel(MoeCombineArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ES = KIND == X_F32 ? 4 : 2, U = 4, N = kCols<KIND>;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= a.T * a.pieces) return;
  const uint32_t t = a.by_pieces.div(i), h = (i - t * a.pieces) * (uint32_t)N, live = a.H - h;
  const int64_t c = (int64_t)t * a.k;
  const uint32_t back = past_end<N>(live);
  float s[N] = {};
  if (a.rows != 0)
    for (uint32_t j0 = 0; j0 < a.k; j0 += U) {
      Run<KIND, N> r[U];
      float f[U];
      bool has[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t j = min(j0 + u, a.k - 1);
        const uint32_t row = (uint32_t)a.row_of[c + j];
        has[u] = j0 + u < a.k && row < a.rows;
        f[u] = weight(a.w, c + j, a.wkind);
        r[u] = load_run<KIND, N, FAR>(a.R + (int64_t)(has[u] ? row : 0u) * a.ldr + (int64_t)h * ES, a.H, back);
      }
      if (back != 0)
#pragma unroll
        for (int u = 0; u < U; ++u) move_down(r[u], back);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[N];
        values_of(v, r[u]);
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = has[u] ? __builtin_fmaf(f[u], v[e], s[e]) : s[e];
      }
    }
  const uint32_t yes = a.ykind == X_F32 ? 4u : 2u;
  if (a.add != nullptr) {
    float v[N];
    const uint8_t* p = a.add + (int64_t)t * a.ldadd + (int64_t)h * yes;
    auto addend = [&](auto kind) {
      constexpr int K = decltype(kind)::value;
      Run<K, N> r = load_run<K, N>(p, a.H, back);
      if (back != 0) move_down(r, back);
      values_of(v, r);
    };
    if (a.ykind == X_F32) addend(std::integral_constant<int, X_F32>{});
    else if (a.ykind == X_BF16) addend(std::integral_constant<int, X_BF16>{});
    else addend(std::integral_constant<int, X_F16>{});
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] += v[e];
  }
  store_values<N, FAR>(a.Y + (int64_t)t * a.ldy + (int64_t)h * yes, s, live, a.ykind);
#endif
}

struct MoeGradArgs {
  const uint8_t* dY;
  const uint8_t* R;
  const uint8_t* w;
  uint8_t* dR;  // null: not wanted
  uint8_t* dw;  // null: not wanted
  const int32_t* row_of;
  int64_t lddy, ldr, lddr;  // bytes
  uint32_t T, k, H, rows;
  uint32_t wkind;
  uint32_t parts;  // tasks of a token
  FastDiv by_parts;
};

// WPT waves, a workgroup, a token (WPT = 1: four tokens a workgroup), or a part of
// its choices: they walk the row together, U choices at a time, each lane 16 bytes
// of dY against the same of each row.  Bound by memory: 8192 x 4 rows of 4096 bf16, 604
// MB, 126 us, 4.8 TB/s; a small one by its chain of loads and the sum over the waves
// (16 x 4 rows of 4096 bf16 5.1 us).
template <int WPT>
constexpr int kGradThreads = WPT == 1 ? 256 : 64 * WPT;
template <int KIND, int WPT, bool FAR>
__global__ void __launch_bounds__(kGradThreads<WPT>) moe_combine_grad_kernel(MoeGradArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ES = KIND == X_F32 ? 4 : 2, U = 4, N = kCols<KIND>;
  constexpr uint32_t kInd = KIND;
  __shared__ float sums[WPT][U];
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
  const uint32_t task = WPT == 1 ? blockIdx.x * 4u + wave : blockIdx.x;
  const uint32_t t = a.by_parts.div(task), part = task - t * a.parts;
  if (t >= a.T) return;  // (whole workgroups where they meet below)
  const int64_t c = (int64_t)t * a.k;
  const uint8_t* dy = a.dY + (int64_t)t * a.lddy;
  for (uint32_t j0 = part * U; j0 < a.k; j0 += a.parts * U) {
    uint32_t row[U];
    float f[U], dot[U];
    bool has[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t j = min(j0 + u, a.k - 1);
      row[u] = (uint32_t)a.row_of[c + j];
      has[u] = j0 + u < a.k && row[u] < a.rows;
      if (!has[u]) row[u] = 0;
      f[u] = weight(a.w, c + j, a.wkind);
      dot[u] = 0.0f;
    }
    if (a.rows != 0)
      for (uint32_t h = (WPT == 1 ? lane : threadIdx.x) * (uint32_t)N; h < a.H; h += WPT * 64u * N) {
        const uint32_t live = a.H - h;
        const int64_t off = (int64_t)h * ES;
        const uint32_t back = past_end<N>(live);
        float g[N];
        Run<KIND, N> y = load_run<KIND, N>(dy + off, a.H, back), r[U];
        if (a.dw != nullptr) {
#pragma unroll
          for (int u = 0; u < U; ++u) r[u] = load_run<KIND, N>(a.R + (int64_t)row[u] * a.ldr + off, a.H, back);
          if (back != 0)
#pragma unroll
            for (int u = 0; u < U; ++u) move_down(r[u], back);
        }
        if (back != 0) move_down(y, back);
        values_of(g, y);
        if (a.dw != nullptr)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[N];
            values_of(v, r[u]);
#pragma unroll
            for (int e = 0; e < N; ++e) dot[u] = __builtin_fmaf(g[e], v[e], dot[u]);
          }
        if (a.dR != nullptr)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (!has[u]) continue;
            float o[N];
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = f[u] * g[e];
            store_values<N, FAR>(a.dR + (int64_t)row[u] * a.lddr + off, o, live, kInd);
          }
      }
    if (a.dw == nullptr) continue;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) dot[u] += __shfl_xor(dot[u], d);
    if constexpr (WPT != 1) {
      if (lane == 0)
#pragma unroll
        for (int u = 0; u < U; ++u) sums[wave][u] = dot[u];
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        dot[u] = sums[0][u];
#pragma unroll
        for (int w = 1; w < WPT; ++w) dot[u] += sums[w][u];
      }
      __syncthreads();
    }
    if ((WPT == 1 ? lane : threadIdx.x) == 0)
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + u < a.k)
          put_value(a.dw + (c + j0 + u) * (a.wkind == X_F32 ? 4 : 2), has[u] ? dot[u] : 0.0f, a.wkind);
  }
#endif
}

}  // namespace bst
