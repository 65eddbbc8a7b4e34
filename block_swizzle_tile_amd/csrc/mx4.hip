// mx4.hip -- host side of the 4-bit operators declared in include/bst_mx4.h:
// argument checks (before any HIP call), the choice of tile and split, and the
// launches.
#include <cmath>

#include "bst_host.hpp"
#include "bst_mx4_instances.hpp"
#include "bst_mx4_quant.hpp"
#include "bst_mx4_rows.hpp"

using namespace bst;
using namespace bst::host;

namespace {

// A matrix of 4-bit codes (pad 16) or of its scales (pad 4), row lengths and
// pitches in bytes.
bst_status bytes_ok(const char* what, const void* p, int64_t ld, int64_t cols, int64_t pad) {
  if (!p) return set_error(BST_E_INVAL, "%s is NULL", what);
  if (ld < cols)
    return set_error(BST_E_INVAL, "%s: leading dimension %lld below the row length %lld", what,
                     (long long)ld, (long long)cols);
  if (!aligned(p, (uint64_t)pad) || ld % pad != 0)
    return set_error(BST_E_ALIGN, "%s: base and leading dimension must be multiples of %lld bytes", what,
                     (long long)pad);
  if (ld > kSpan || 256 * ld + 128 >= kSpan)
    return set_error(BST_E_UNSUPPORTED, "%s: 256 rows of pitch %lld span 2 GiB", what, (long long)ld);
  return BST_OK;
}

// Tile, split and form of a product.  count: groups (0: plain).
//
// What is not asked for is the pair of least cost, in microseconds, of a model
// that was fitted to times of all tiles: a round of workgroups costs a tile's
// start and end, and its stages, both more where all CUs load and store at once;
// a split adds a launch and its partial sums, written and read at 5 TB/s; groups take
// what reading their weights does (1000 rows over 16 groups of 4096 x 4096: 51.5 us
// with 32 rows a tile, 41.7 with 64, 29.8 with 128).  The choice is within 5% of the
// best of all tiles and splits 1 to 8 in 54 of 60 drawn shapes (8 to 4096 rows, 256 to
// 8192 columns, K 256 to 8192) and within 10% in 59; of all tiles in 66 and 74 of 80
// drawn grouped shapes (the worst: 8192 rows over 32 groups of 2048 x 2048, 47.4 us
// for 38.7).
struct Mx4Plan : Plan {
  int stages = 0;
};

bst_status plan_mx4(int64_t count, int64_t M, int64_t N, int64_t K, const Sched& s, Mx4Plan& p) {
  struct Tile {
    uint32_t m, n;
    int stages;
    double ends[2], stage[2];  // with few CUs at work, with all
  };
  // (of two stages below 256x256: a pair of workgroups, which share a CU)
  static constexpr Tile kTiles[] = {{32, 128, 4, {2.2, 3.0}, {0.20, 0.23}},  {32, 128, 2, {2.8, 2.8}, {0.65, 0.65}},
                                    {64, 128, 4, {2.2, 3.2}, {0.25, 0.35}},  {64, 128, 2, {2.7, 2.7}, {0.73, 0.73}},
                                    {128, 128, 4, {2.4, 3.5}, {0.28, 0.64}}, {128, 128, 2, {3.8, 3.8}, {1.15, 1.15}},
                                    {256, 256, 2, {4.2, 7.0}, {0.85, 1.69}}};
  const int64_t cus = device_cu_count(), nk = cdiv(K, kMx4Stage);
  const int64_t groups = count ? std::max<int64_t>(std::min(count, M), 1) : 1;
  if (count && s.split > 1) return set_error(BST_E_UNSUPPORTED, "grouped products are not split");
  double best = -1;
  for (const Tile& t : kTiles) {
    if ((s.tm != 0 || s.tn != 0) && (s.tm != t.m || s.tn != t.n)) continue;
    // tiles at most, and those that groups of one size would have: half a tile more
    // than their rows fill
    const int64_t most = (count ? cdiv(M, t.m) + count : cdiv(M, t.m)) * cdiv(N, t.n);
    const double each = (double)M / groups / t.m;  // tiles that a group's rows fill
    const double rows = groups > 1 ? groups * std::max(1.0, each + 0.5) : (double)cdiv(M, t.m);
    const double tiles = std::max(1.0, rows * cdiv(N, t.n));
    const bool paired = t.stages == 2 && t.m < 256;
    const int64_t from = s.split ? s.split : 1, to = s.split ? s.split : count || tiles >= cus ? 1 : std::min<int64_t>(nk, 16);
    for (int64_t n = from; n <= std::max(from, to); ++n) {
      const int64_t ks = nk ? cdiv(nk, n) : 0, slices = nk ? cdiv(nk, ks) : 1;  // no empty slice
      const double work = tiles * slices / cus, load = std::min(1.0, work);
      if (t.m < 256 && paired != (work > 1)) continue;
      // (a workgroup that has a CU to itself takes two thirds of a pair's time)
      const double pairs = std::floor(std::ceil(work) / 2), odd = std::ceil(work) - 2 * pairs;
      const double rounds = paired ? pairs + 0.65 * odd : std::ceil(work);
      const double cost = rounds * (t.ends[0] + (t.ends[1] - t.ends[0]) * load +
                                    ks * (t.stage[0] + (t.stage[1] - t.stage[0]) * load)) +
                          (slices > 1 ? 2.5 + slices * (double)M * N * 8 / 5e6 : 0);
      // weights that no L2 holds (a group's last rows come long after its whole tiles,
      // and read them again)
      const double bytes = groups > 1 ? (double)groups * N * K * 0.53 : 0;
      const double weights = bytes < 32e6 ? 0 : (each < 0.7 ? 1.0 : each < 1.4 ? 1.5 : 2.0) * bytes / 5.2e6 + 4;
      if (best >= 0 && std::max(cost, weights) >= best) continue;
      best = std::max(cost, weights);
      p.tm = t.m;
      p.tn = t.n;
      p.tiles = most;
      p.split = (uint32_t)slices;
      p.stages = t.stages;
    }
  }
  if (best < 0) return set_error(BST_E_UNSUPPORTED, "no 4-bit kernel with tile %ux%u", s.tm, s.tn);
  return plan_workspace(p, M, N);
}

// 16-row fragments of the kernel for a few rows (count: groups, 0: plain), or 0
// where the tiles take the product: where a tile or a split is asked for, where
// K is long (a workgroup walks all of it), or where there are more workgroups of
// 16 columns than the chip holds at once, of which each reads all rows of A.
// Times in us against the best tile, M x N x K:
//   1 x 4096 x 4096 4.7 / 7.3, 1 x 4096 x 14336 9.1 / 11.6, 1 x 16384 x 4096
//   10.6 / 9.2 (left to the tiles), 16 x 1024 x 28672 20.9 / 13.5 (left), 32 x
//   4096 x 4096 7.0 / 8.0, 32 x 8192 x 2048 7.6 / 6.2 (left), 64 x 1024 x 1024
//   4.2 / 5.0, 64 x 4096 x 4096 10.0 / 8.0 (left); groups: 16 rows of 16 groups,
//   256 x 3360 4.3 / 9.9, 58 of 7, 1152 x 992 4.8 / 7.0, 64 of 32, 2048 x 4096
//   33.4 / 25.6 (left).
// How even the groups' loads are is not known here.  A group of more than 16 f rows has
// further workgroups: 192 rows over 8 groups of 512 x 7168 take 9.1 / 11.1 with 24 rows
// each, 13.8 / 11.3 with up to 44 and 10.5 / 11.3 with all in one; 512 over 64 of 128 x
// 1024 4.2 / 6.4, 5.9 / 6.4 and 4.6 / 6.5.  The worst of 15 sizes with loads of four
// kinds: 15.8 / 11.3.
int row_fragments(int64_t count, int64_t M, int64_t N, int64_t K, const Sched& s) {
  if (s.tm != 0 || s.tn != 0 || s.split > (count ? 1u : 0u)) return 0;
  const int64_t per = count ? cdiv(M, count) : M;  // rows of a group, on average
  if (per > (count ? 24 : 64)) return 0;
  const int64_t f = count ? (per <= 8 ? 1 : 2) : M <= 16 ? 1 : M <= 32 ? 2 : 4;
  const int64_t tiles = cdiv(N, 16) * std::max<int64_t>(count, 1);
  return f * cdiv(K, kMx4Stage) <= 56 && f * tiles <= 2 * device_cu_count() ? (int)f : 0;
}

bst_status gemm(bst_dtype c, bool grouped, int32_t G, const int32_t* group_m, int64_t M, int64_t N, int64_t K,
                const uint8_t* A, int64_t lda, const uint8_t* SA, int64_t ldsa, const uint8_t* B, int64_t ldb,
                int64_t strideB, const uint8_t* SB, int64_t ldsb, int64_t strideSB, void* C, int64_t ldc,
                const bst_sched* sched, void* ws, size_t ws_bytes, void* stream) {
  bst_status st = sizes_ok(M, N, K);
  if (st != BST_OK) return st;
  if (!out_bytes(c)) return set_error(BST_E_UNSUPPORTED, "output dtype %d", (int)c);
  if (grouped && (st = groups_ok(G, group_m)) != BST_OK) return st;
  Sched s;
  if ((st = read_sched(sched, kMx4Stage, s)) != BST_OK) return st;
  if (M == 0 || N == 0) return BST_OK;
  if ((st = matrix_ok("C", C, ldc, N, out_bytes(c))) != BST_OK) return st;
  const int64_t kq = cdiv(K, 2), kb = cdiv(K, 32);
  if (K > 0) {
    if ((st = bytes_ok("A", A, lda, kq, 16)) != BST_OK) return st;
    if ((st = bytes_ok("B", B, ldb, kq, 16)) != BST_OK) return st;
    if ((st = bytes_ok("scale_a", SA, ldsa, kb, 4)) != BST_OK) return st;
    if ((st = bytes_ok("scale_b", SB, ldsb, kb, 4)) != BST_OK) return st;
    if (grouped && (strideB < 0 || strideSB < 0)) return set_error(BST_E_INVAL, "negative group stride");
    if (grouped && (strideB % 16 != 0 || strideSB % 4 != 0))
      return set_error(BST_E_ALIGN, "strideB must be a multiple of 16 bytes, strideSB of 4");
  }
  const int rows = row_fragments(grouped ? G : 0, M, N, K, s);
  Mx4Plan p;
  if (!rows) {
    if ((st = plan_mx4(grouped ? G : 0, M, N, K, s, p)) != BST_OK) return st;
    if ((st = check_ws(p, ws, ws_bytes)) != BST_OK) return st;
  }
  const Mx4GemmList l = grouped ? mx4_gemm_grouped() : mx4_gemm_plain();
  const Mx4GemmInstance* in = nullptr;
  for (int i = 0; i < l.count && !in; ++i)
    if ((uint32_t)l.begin[i].bm == p.tm && (uint32_t)l.begin[i].bn == p.tn && l.begin[i].stages == p.stages)
      in = l.begin + i;
  if (!in && !rows) return set_error(BST_E_UNSUPPORTED, "no 4-bit kernel with tile %ux%u", p.tm, p.tn);

  Mx4GemmArgs a{};
  a.A = A;
  a.B = B;
  a.C = static_cast<uint8_t*>(C);
  a.sa = SA;
  a.sb = SB;
  a.lda = lda;
  a.ldb = ldb;
  a.ldsa = ldsa;
  a.ldsb = ldsb;
  a.ldc = ldc;
  a.strideB = strideB;
  a.strideSB = strideSB;
  a.group_m = group_m;
  a.G = (uint32_t)G;
  a.M = (uint32_t)M;
  a.N = (uint32_t)N;
  a.K = (uint32_t)K;
  a.nk = (uint32_t)cdiv(K, kMx4Stage);
  a.kslice = (uint32_t)cdiv(a.nk, p.split);
  a.tiles = (uint32_t)p.tiles;
  a.off = s.off;
  a.dir = s.dir;
  a.remap = s.remap;
  a.grid = (uint32_t)(p.tiles * p.split);
  a.ckind = (uint32_t)c;
  // a tile's rows of C are stored at 31-bit offsets
  a.cvec = vec_rows(C, ldc, 0, out_bytes(c)) && 256 * ldc * out_bytes(c) < kSpan;
  a.far = is_far(M, N * out_bytes(c), 4 * kFar);
  if (rows) {
    // behind each group's first rows: at most a part for every 16 `rows` of the rest
    const dim3 grid((uint32_t)(cdiv(N, 16) * (grouped ? G + M / (16 * rows) : 1))), block(512);
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, (hipStream_t)stream, a);
      return launched(hipGetLastError(), "4-bit product");
    };
    if (grouped) return rows == 1 ? run(mx4_rows_kernel<1, 4, true>) : run(mx4_rows_kernel<2, 4, true>);
    if (rows == 1) return run(mx4_rows_kernel<1, 4, false>);
    return rows == 2 ? run(mx4_rows_kernel<2, 4, false>) : run(mx4_rows_kernel<4, 2, false>);
  }
  if (p.split > 1) {
    a.part = static_cast<float*>(ws);
    a.pitch = p.pitch;
  }
  if (!grouped)
    a.mc = make_map_consts((uint32_t)cdiv(M, p.tm), (uint32_t)cdiv(N, p.tn), s.off, s.dir, (uint32_t)p.tiles,
                           a.kslice);
  st = launched(in->launch(a.grid, (hipStream_t)stream, a), "4-bit product");
  if (st != BST_OK || p.split == 1) return st;
  return reduce(p, 1, M, N, a.part, C, ldc, 0, nullptr, 0, 0, c, stream);
}

// What the quantiser and its inverse check alike; rows x cols: of Q, in values.
bst_status quant_args(Mx4QuantArgs& a, bst_dtype x, int64_t M, int64_t K, int64_t rows, int64_t cols,
                      int64_t ldx, int64_t ldq, int64_t lds) {
  bst_status st = sizes_ok(M, 0, K);
  if (st != BST_OK) return st;
  if (!out_bytes(x)) return set_error(BST_E_UNSUPPORTED, "dtype %d", (int)x);
  const int64_t kb = cdiv(cols, 32);
  if (ldx < K || ldq < cdiv(cols, 2) || lds < kb)
    return set_error(BST_E_INVAL, "leading dimension too small (ldx %lld, ldq %lld, lds %lld for %lld x %lld)",
                     (long long)ldx, (long long)ldq, (long long)lds, (long long)M, (long long)K);
  if (ldx > kSpan || ldq > kSpan || lds > kSpan) return set_error(BST_E_INVAL, "leading dimension above 2^31");
  if (rows > 0 && kb > kMaxSize / rows) return set_error(BST_E_INVAL, "more than 2^31-1 blocks");
  a.ldx = ldx;
  a.ldq = ldq;
  a.lds = lds;
  a.M = (uint32_t)M;
  a.K = (uint32_t)K;
  a.kb = (uint32_t)kb;
  a.blocks = (uint32_t)(rows * kb);
  a.by_kb = make_fastdiv((uint32_t)std::max<int64_t>(kb, 1));
  return BST_OK;
}

// go(type, yes or no) with both known at compile time.
template <typename F>
bst_status for_values(bst_dtype x, bool yes, F&& go) {
  auto with = [&](auto kind) {
    return yes ? go(kind, std::bool_constant<true>{}) : go(kind, std::bool_constant<false>{});
  };
  if (x == BST_F32) return with(std::integral_constant<int, X_F32>{});
  return x == BST_BF16 ? with(std::integral_constant<int, X_BF16>{}) : with(std::integral_constant<int, X_F16>{});
}

// Workgroups that take `per` blocks each and step.
uint32_t row_grid(uint32_t blocks, int64_t per) {
  return (uint32_t)std::min<int64_t>(cdiv(blocks, per), (int64_t)device_cu_count() * 64);
}

}  // namespace

extern "C" {

bst_status bst_quant_mx4(bst_dtype x, int64_t M, int64_t K, int32_t transpose, const void* X, int64_t ldx,
                         uint8_t* Q, int64_t ldq, uint8_t* S, int64_t lds, void* stream) {
  if (transpose != 0 && transpose != 1) return set_error(BST_E_INVAL, "transpose must be 0 or 1");
  Mx4QuantArgs a{};
  bst_status st = transpose ? quant_args(a, x, M, K, K, M, ldx, ldq, lds)
                            : quant_args(a, x, M, K, M, K, ldx, ldq, lds);
  if (st != BST_OK) return st;
  if (M == 0 || K == 0) return BST_OK;
  if (!X || !Q || !S) return set_error(BST_E_INVAL, "X, Q or S is NULL");
  if (!aligned(X, (uint64_t)out_bytes(x))) return set_error(BST_E_ALIGN, "X is not aligned to its type");
  a.X = static_cast<const uint8_t*>(X);
  a.Q = Q;
  a.S = S;
  auto run = [&](auto kernel, int64_t grid, uint32_t threads = 256) {
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(threads), 0, (hipStream_t)stream, a);
    return launched(hipGetLastError(), "4-bit quantisation");
  };
  if (transpose) {
    const bool much = is_far(M, K * out_bytes(x), 4 * kFar);
    const int64_t nb = much ? 8 : 4, grid = cdiv(K, 128) * cdiv(a.kb, nb);
    if ((st = grid_ok(grid, 64 * nb)) != BST_OK) return st;
    return for_values(x, much, [&](auto k, auto m) {
      return run(mx4_quant_cols<k.value, m.value ? 8 : 4>, grid, 64 * (uint32_t)nb);
    });
  }
  const int64_t grid = row_grid(a.blocks, 64);
  if (x == BST_F32) return run(mx4_quant_rows<X_F32>, grid);
  return x == BST_BF16 ? run(mx4_quant_rows<X_BF16>, grid) : run(mx4_quant_rows<X_F16>, grid);
}

bst_status bst_dequant_mx4(bst_dtype x, int64_t M, int64_t K, const uint8_t* Q, int64_t ldq, const uint8_t* S,
                           int64_t lds, void* X, int64_t ldx, void* stream) {
  Mx4QuantArgs a{};
  bst_status st = quant_args(a, x, M, K, M, K, ldx, ldq, lds);
  if (st != BST_OK) return st;
  if (M == 0 || K == 0) return BST_OK;
  if (!X || !Q || !S) return set_error(BST_E_INVAL, "X, Q or S is NULL");
  if (!aligned(X, (uint64_t)out_bytes(x))) return set_error(BST_E_ALIGN, "X is not aligned to its type");
  a.Xo = static_cast<uint8_t*>(X);
  a.Q = const_cast<uint8_t*>(Q);
  a.S = const_cast<uint8_t*>(S);
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(row_grid(a.blocks, x == BST_F32 ? 32 : 64)), dim3(256), 0, (hipStream_t)stream, a);
    return launched(hipGetLastError(), "4-bit restoring");
  };
  return for_values(x, is_far(M, K * out_bytes(x), 4 * kFar),
                    [&](auto k, auto f) { return run(mx4_dequant<k.value, f.value>); });
}

bst_status bst_gemm_mx4(bst_dtype c, int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda,
                        const uint8_t* SA, int64_t ldsa, const uint8_t* B, int64_t ldb, const uint8_t* SB,
                        int64_t ldsb, void* C, int64_t ldc, const bst_sched* sched, void* ws, size_t ws_bytes,
                        void* stream) {
  return gemm(c, false, 1, nullptr, M, N, K, A, lda, SA, ldsa, B, ldb, 0, SB, ldsb, 0, C, ldc, sched, ws,
              ws_bytes, stream);
}

bst_status bst_grouped_gemm_mx4(bst_dtype c, int32_t G, const int32_t* group_m, int64_t total_m, int64_t N,
                                int64_t K, const uint8_t* A, int64_t lda, const uint8_t* SA, int64_t ldsa,
                                const uint8_t* B, int64_t ldb, int64_t strideB, const uint8_t* SB,
                                int64_t ldsb, int64_t strideSB, void* C, int64_t ldc, const bst_sched* sched,
                                void* stream) {
  return gemm(c, true, G, group_m, total_m, N, K, A, lda, SA, ldsa, B, ldb, strideB, SB, ldsb, strideSB, C,
              ldc, sched, nullptr, 0, stream);
}

size_t bst_mx4_workspace_bytes(int64_t M, int64_t N, int64_t K, const bst_sched* sched) {
  Sched s;
  Mx4Plan p;
  if (sizes_ok(M, N, K) != BST_OK || read_sched(sched, kMx4Stage, s) != BST_OK) return 0;
  if (row_fragments(0, M, N, K, s)) return 0;
  return plan_mx4(0, M, N, K, s, p) == BST_OK ? p.ws : 0;
}

}  // extern "C"
