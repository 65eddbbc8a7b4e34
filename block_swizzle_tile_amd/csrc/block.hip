// block.hip -- host side of the block-scaled operators declared in
// include/bst_block.h: argument checks (before any HIP call), the choice of
// tile and split, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bst_block_instances.hpp"
#include "bst_block_quant.hpp"

using namespace bst;

namespace {

constexpr int64_t kMaxSize = 0x7fffffffLL;
constexpr int64_t kSpan = 1LL << 31;  // reach of a panel's byte offsets

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, uint64_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int out_bytes(bst_dtype t) {
  return t == BST_F32 ? 4 : t == BST_F16 || t == BST_BF16 ? 2 : 0;
}
int scale_bytes(bst_dtype t) { return t == BST_F32 ? 4 : t == BST_E8M0 ? 1 : 0; }

// Rows of `t` at p with pitch ld take 16-byte accesses.
bool vec_rows(const void* p, int64_t ld, int64_t stride, int es) {
  return aligned(p, 16) && ld * es % 16 == 0 && stride * es % 16 == 0;
}

bst_status sizes_ok(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return set_error(BST_E_INVAL, "negative size");
  if (M > kMaxSize || N > kMaxSize || K > kMaxSize)
    return set_error(BST_E_INVAL, "size above 2^31-1");
  return BST_OK;
}

bst_status groups_ok(int32_t G, const int32_t* group_m) {
  if (G < 1 || G > kMaxGroups)
    return set_error(BST_E_INVAL, "group count %d outside [1, %d]", (int)G, kMaxGroups);
  if (!group_m) return set_error(BST_E_INVAL, "group sizes are NULL");
  if (!aligned(group_m, 4)) return set_error(BST_E_ALIGN, "group sizes are not 4-byte aligned");
  return BST_OK;
}

// A matrix of 8-bit codes: rows of whole 16-byte chunks.
bst_status codes_ok(const char* what, const void* p, int64_t ld, int64_t cols, int64_t tile_rows) {
  if (!p) return set_error(BST_E_INVAL, "%s is NULL", what);
  if (ld < cols)
    return set_error(BST_E_INVAL, "%s: leading dimension %lld below the row length %lld", what,
                     (long long)ld, (long long)cols);
  if (!aligned(p, 16) || ld % 16 != 0)
    return set_error(BST_E_ALIGN, "%s: base and leading dimension must be multiples of 16 bytes",
                     what);
  if (ld > kSpan || tile_rows * ld + 128 >= kSpan)
    return set_error(BST_E_UNSUPPORTED, "%s: %lld rows of pitch %lld span 2 GiB", what,
                     (long long)tile_rows, (long long)ld);
  return BST_OK;
}

bst_status scales_ok(const char* what, const void* p, bst_dtype t, int64_t ld, int64_t cols) {
  const int b = scale_bytes(t);
  if (b == 0) return set_error(BST_E_UNSUPPORTED, "%s: scale type %d is neither E8M0 nor F32", what, (int)t);
  if (!p) return set_error(BST_E_INVAL, "%s is NULL", what);
  if (ld < cols)
    return set_error(BST_E_INVAL, "%s: leading dimension %lld below the row length %lld", what,
                     (long long)ld, (long long)cols);
  if (!aligned(p, (uint64_t)b)) return set_error(BST_E_ALIGN, "%s is not aligned to its type", what);
  if (ld > kSpan || 256 * ld * b >= kSpan)
    return set_error(BST_E_UNSUPPORTED, "%s: 256 rows of pitch %lld span 2 GiB", what, (long long)ld);
  return BST_OK;
}

bst_status matrix_ok(const char* what, const void* p, int64_t ld, int64_t cols, int es) {
  if (!p) return set_error(BST_E_INVAL, "%s is NULL", what);
  if (ld < cols)
    return set_error(BST_E_INVAL, "%s: leading dimension %lld below the row length %lld", what,
                     (long long)ld, (long long)cols);
  if (ld > kSpan) return set_error(BST_E_INVAL, "%s: leading dimension above 2^31", what);
  if (!aligned(p, (uint64_t)es)) return set_error(BST_E_ALIGN, "%s is not aligned to its type", what);
  return BST_OK;
}

bst_status launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return BST_OK;
  return set_error(BST_E_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
}

// A launch holds fewer than 2^32 threads.
bool grid_fits(int64_t workgroups, int64_t threads) { return workgroups <= 0xffffffffLL / threads; }
bst_status grid_ok(int64_t workgroups, int64_t threads) {
  if (grid_fits(workgroups, threads)) return BST_OK;
  return set_error(BST_E_UNSUPPORTED, "%lld workgroups of %lld threads are more than one launch holds",
                   (long long)workgroups, (long long)threads);
}

// ------------------------------------------------------------ schedule ----
struct Sched {
  uint32_t tm = 0, tn = 0, off = 8, dir = BST_ZN, remap = 1, split = 0;
};

bst_status read_sched(const bst_sched* s, uint32_t tile_k, Sched& d) {
  if (!s) return BST_OK;
  if (s->swizzle_offset == 0) return set_error(BST_E_INVAL, "swizzle_offset must be >= 1");
  if (s->swizzle_direction > 2)
    return set_error(BST_E_INVAL, "swizzle_direction %u not in {0 Zn, 1 Nz, 2 raster}",
                     s->swizzle_direction);
  if (s->xcd_remap > 1) return set_error(BST_E_INVAL, "xcd_remap must be 0 or 1");
  if (s->split_k > 64) return set_error(BST_E_INVAL, "split_k %u above 64", s->split_k);
  if (s->tile_k != 0 && s->tile_k != tile_k)
    return set_error(BST_E_UNSUPPORTED, "tile_k %u is not provided", s->tile_k);
  if (s->grid || s->path || s->shuffle_k || s->dynamic || s->preload)
    return set_error(BST_E_UNSUPPORTED,
                     "grid, path, shuffle_k, dynamic and preload must be 0 for block-scaled calls");
  d.tm = s->tile_m;
  d.tn = s->tile_n;
  d.off = s->swizzle_offset;
  d.dir = s->swizzle_direction;
  d.remap = s->xcd_remap;
  d.split = s->split_k;
  return BST_OK;
}

struct Plan {
  uint32_t tm = 0, tn = 0, split = 1, pitch = 0;
  int64_t tiles = 0;  // per slice (a bound when grouped)
  size_t ws = 0;
};

// Partial sums: a slice's rows x pitch floats, rows of whole 16 bytes.
bst_status plan_workspace(Plan& p, int64_t rows, int64_t N) {
  p.pitch = (uint32_t)(cdiv(N, 4) * 4);
  if (p.split > 1) {
    // sum_partials counts quads, and a grid's worth past the last, in 32 bits
    if (rows > kMaxSize / std::max<int64_t>(p.pitch / 4, 1))
      return set_error(BST_E_INVAL, "a split output of %lld rows of %lld is too large",
                       (long long)rows, (long long)N);
    p.ws = (size_t)p.split * (size_t)rows * p.pitch * 4;
  }
  return grid_ok(p.tiles * p.split, 512);
}

// Tile and split of a product.  count: groups (0: plain); exact: an fp32 output.
// The large tile goes by all rows, also where a group's rows fill half of it:
// its longer reuse of the weights outweighs the idle half (8192 rows over 64
// groups, N 4096, K 2048, E8M0: 256x256 166 us, 128x128 200, 64x128 279; N 2048,
// K 4096: 180, 183, 245; over 8 groups of N 4096, K 2048: 86, 126, 182).
bst_status plan_gemm(int64_t count, int64_t M, int64_t N, int64_t K, bool exact, const Sched& s,
                     Plan& p) {
  const int64_t cus = device_cu_count(), G = std::max<int64_t>(count, 1);
  const int64_t per = cdiv(M, G);  // rows of a group, on average
  auto tiles = [&](int64_t tm, int64_t tn) {
    return (count ? cdiv(M, tm) + G : cdiv(M, tm)) * cdiv(N, tn);
  };
  p.tm = s.tm;
  p.tn = s.tn;
  if (p.tm == 0 && p.tn == 0) {
    p.tn = 128;
    if (per <= 32) p.tm = 32;
    else if (per <= 64) p.tm = 64;
    else if (!exact && cdiv(M, 256) * cdiv(N, 256) * 4 >= cus * 3) p.tm = p.tn = 256;
    else if (cdiv(M, 128) * cdiv(N, 128) * 4 >= cus * 3) p.tm = 128;
    else p.tm = 64;
  }
  const bool known = (p.tn == 128 && (p.tm == 32 || p.tm == 64 || p.tm == 128)) ||
                     (p.tm == 256 && p.tn == 256 && !exact);
  if (!known)
    return set_error(BST_E_UNSUPPORTED, "no block-scaled kernel with tile %ux%u%s", p.tm, p.tn,
                     exact ? " and an fp32 output" : "");
  p.tiles = tiles(p.tm, p.tn);
  const int64_t nk = cdiv(K, 128);
  int64_t split = s.split;
  if (count) {
    if (split > 1) return set_error(BST_E_UNSUPPORTED, "grouped products are not split");
    split = 1;
  } else if (split == 0) {
    split = 1;
    // one workgroup per CU: beyond that a split only adds partial sums (one row
    // on the 32x128 tile, 4096 x 4096: 10.3 us at half the CUs, 9.2 at all, 13.4
    // at twice)
    if (p.tiles > 0 && p.tiles < cus && nk >= 4)
      split = std::max<int64_t>(1, std::min<int64_t>({cus / p.tiles, nk / 2, 16}));
  }
  if (nk == 0) split = 1;
  const int64_t ks = nk ? cdiv(nk, split) : 0;
  p.split = (uint32_t)(nk ? cdiv(nk, ks) : 1);  // no empty slice
  return plan_workspace(p, M, N);
}

// Tile and split (along the rows) of a weight gradient; parts: bf16 parts of dY
// (1 to 3).  What is not asked for is the pair of least cost, in microseconds,
// of a model with three terms: a stage of 64 rows takes as long as the table
// says (one workgroup per CU; two take twice as long), a slice's partial sums
// are written and read once at 5 TB/s, and adding them is one launch more.
// Against the best of both tiles and splits 1 to 32 the choice is within 10%
// over 64 .. 8192 rows and weights from 64 x 64 to 4096 x 4096 in 16 of 17
// shapes (16384 rows, 1024 x 1024: 61.0 us against 52.8); the types' own costs
// matter with fp16 and fp32 gradients (4096 rows, 2048 x 2048: fp32 171 us on
// 128x128 unsplit, 130 on 256x256 cut four ways; fp16 129 and 99).
bst_status plan_grad(int64_t count, int64_t M, int64_t N, int64_t K, int parts, const Sched& s,
                     Plan& p) {
  static constexpr double kStage[3][2] = {{0.75, 1.75}, {1.95, 4.7}, {2.6, 6.2}};
  const int64_t cus = device_cu_count(), G = std::max<int64_t>(count, 1);
  if (!(s.tm == s.tn && (s.tm == 0 || s.tm == 128 || s.tm == 256)))
    return set_error(BST_E_UNSUPPORTED, "no weight-gradient kernel with tile %ux%u", s.tm, s.tn);
  const int64_t stages = std::max<int64_t>(cdiv(cdiv(M, G), 64), 1);
  const double slice = (double)G * K * N * 8 / 5e6 + 0.07;
  double best = -1;
  int64_t fewest = 0;
  for (int64_t tile = 128; tile <= 256; tile += 128) {
    if (s.tm != 0 && s.tm != tile) continue;
    const int64_t tiles = G * cdiv(K, tile) * cdiv(N, tile);
    fewest = tiles;
    if (!grid_fits(tiles, 512)) continue;  // 64 times the others stay in 64 bits
    const double stage = kStage[parts - 1][tile / 256];
    for (int64_t n = 1; n <= std::min<int64_t>(s.split ? s.split : 32, stages); ++n) {
      if (s.split && n != std::min<int64_t>(s.split, stages)) continue;
      const double cost = (double)cdiv(tiles * n, cus) * cdiv(stages, n) * stage +
                          (n > 1 ? n * slice + 2 : 0);
      if (best < 0 || cost < best) {
        best = cost;
        p.tm = p.tn = (uint32_t)tile;
        p.tiles = tiles;
        p.split = (uint32_t)n;
      }
    }
  }
  if (best < 0) return grid_ok(fewest, 512);
  return plan_workspace(p, G * K, N);
}

// Products that the kernels for a few rows take, if no tile and no split is
// asked for.  They need one launch and no partial sums, but a workgroup walks
// all of K and reads all of A, so they lose to a split where K is long or the
// rows are many, and to unsplit tiles where the columns are many.  Times in us,
// these kernels against the tiles, M x N x K (sizes that the rule leaves to the
// tiles among them):
// N x K weights: 1 x 4096 x 4096 5.2 / 9.2, 1 x 4096 x 14336 12.8 / 14.6,
//   16 x 4096 x 6144 8.9 / 9.9, 16 x 4096 x 8192 12.2 / 10.5,
//   32 x 4096 x 2944 7.3 / 9.9, 32 x 4096 x 4096 10.6 / 10.0,
//   1 x 1024 x 8192 7.6 / 8.1, 1 x 2048 x 14336 10.7 / 11.3, 1 x 256 x 4096
//   4.6 / 7.5, 1 x 16384 x 4096 16.0 / 14.8; the rule loses where a row's K is
//   longer still and the columns are few: 1 x 512 x 16384 11.5 / 10.3,
//   1 x 1024 x 28672 18.6 / 13.9, 1 x 512 x 32768 20.6 / 14.2;
// K x N weights: 1 x 4096 x 4096 7.2 / 7.9, 1 x 4096 x 8192 14.1 / 9.8,
//   32 x 8192 x 2048 6.9 / 9.9, 33 x 4112 x 2056 6.4 / 9.7,
//   33 x 4096 x 4096 11.7 / 10.5, 1 x 14336 x 2048 10.6 / 8.9; few columns:
//   1 x 256 x 4096 5.7 / 7.3, 32 x 256 x 4096 9.1 / 8.2 (a loss of the rule),
//   64 x 512 x 2944 9.8 / 9.6.
bool takes_rows(int32_t trans_b, int64_t M, int64_t N, int64_t K, const Sched& s) {
  if (s.tm != 0 || s.tn != 0 || s.split != 0) return false;
  const int64_t nk = cdiv(K, 128), cus = device_cu_count();
  if (trans_b)
    return M <= 32 && M * nk <= 768 && cdiv(N, 128) * 2 < cus;
  constexpr int64_t most = BlockRowsN<1, false>::MOST;
  return M <= 64 && nk <= (M <= 32 ? most : most * 3 / 4) && cdiv(N, 32) <= cus;
}

bst_status check_ws(const Plan& p, const void* ws, size_t bytes) {
  if (p.ws == 0) return BST_OK;
  if (!ws || bytes < p.ws)
    return set_error(BST_E_WORKSPACE, "split %u needs %zu workspace bytes (got %zu)", p.split, p.ws,
                     ws ? bytes : (size_t)0);
  if (!aligned(ws, 16)) return set_error(BST_E_ALIGN, "workspace not 16-byte aligned");
  return BST_OK;
}

bst_status reduce(const Plan& p, int64_t count, int64_t rows, int64_t N, const float* part,
                  void* dst, int64_t ld, int64_t stride, const void* add, int64_t ldadd,
                  int64_t strideadd, bst_dtype kind, void* stream) {
  ReduceArgs r{};
  r.part = part;
  r.dst = static_cast<uint8_t*>(dst);
  r.add = static_cast<const uint8_t*>(add);
  r.ld = ld;
  r.stride = stride;
  r.ldadd = ldadd;
  r.strideadd = strideadd;
  r.split = p.split;
  r.rows = (uint32_t)rows;
  r.cols = (uint32_t)N;
  r.pitch = p.pitch;
  r.kind = (uint32_t)kind;
  r.vec = vec_rows(dst, ld, stride, out_bytes(kind)) &&
          (!add || vec_rows(add, ldadd, strideadd, out_bytes(kind)));
  r.quads = make_fastdiv(p.pitch / 4);
  r.by_rows = make_fastdiv((uint32_t)rows);
  r.total = (uint32_t)(count * rows * (p.pitch / 4));
  const uint32_t grid = (uint32_t)std::min<int64_t>(cdiv(r.total, 256), 8192);
  hipLaunchKernelGGL(sum_partials, dim3(grid), dim3(256), 0, (hipStream_t)stream, r);
  return launched(hipGetLastError(), "partial sum");
}

bst_status gemm(bst_dtype c, int32_t trans_b, bool grouped, int32_t G, const int32_t* group_m,
                int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, bst_dtype sa,
                const void* SA, int64_t ldsa, const uint8_t* B, int64_t ldb, int64_t strideB,
                bst_dtype sb, const void* SB, int64_t ldsb, int64_t strideSB, void* C, int64_t ldc,
                const bst_sched* sched, void* ws, size_t ws_bytes, void* stream) {
  bst_status st = sizes_ok(M, N, K);
  if (st != BST_OK) return st;
  if (!out_bytes(c)) return set_error(BST_E_UNSUPPORTED, "output dtype %d", (int)c);
  if (trans_b != 0 && trans_b != 1) return set_error(BST_E_INVAL, "trans_b must be 0 or 1");
  if (grouped && (st = groups_ok(G, group_m)) != BST_OK) return st;
  Sched s;
  if ((st = read_sched(sched, 128, s)) != BST_OK) return st;
  if (M == 0 || N == 0) return BST_OK;
  if ((st = matrix_ok("C", C, ldc, N, out_bytes(c))) != BST_OK) return st;
  const int64_t nk = cdiv(K, 128), nn = cdiv(N, 128);
  if (!scale_bytes(sa) || !scale_bytes(sb))
    return set_error(BST_E_UNSUPPORTED, "a scale type is neither E8M0 nor F32");
  if (K > 0) {
    if ((st = codes_ok("A", A, lda, K, 256)) != BST_OK) return st;
    if ((st = codes_ok("B", B, ldb, trans_b ? K : N, trans_b ? 256 : 128)) != BST_OK) return st;
    if ((st = scales_ok("scale_a", SA, sa, ldsa, nk)) != BST_OK) return st;
    if ((st = scales_ok("scale_b", SB, sb, ldsb, trans_b ? nk : nn)) != BST_OK) return st;
    if (grouped && (strideB < 0 || strideSB < 0))
      return set_error(BST_E_INVAL, "negative group stride");
    if (grouped && strideB % 16 != 0)
      return set_error(BST_E_ALIGN, "strideB must be a multiple of 16 bytes");
  }
  const bool rows = !grouped && takes_rows(trans_b, M, N, K, s);
  Plan p;
  if (!rows) {
    if ((st = plan_gemm(grouped ? G : 0, M, N, K, c == BST_F32, s, p)) != BST_OK) return st;
    if ((st = check_ws(p, ws, ws_bytes)) != BST_OK) return st;
  }
  const int mode = c == BST_F32 ? MODE_EXACT : sa == BST_E8M0 && sb == BST_E8M0 ? MODE_E8M0 : MODE_F32;
  const BlockGemmList l = grouped ? (trans_b ? block_gemm_grouped_t() : block_gemm_grouped_n())
                                  : (trans_b ? block_gemm_plain_t() : block_gemm_plain_n());
  const BlockGemmInstance* in = nullptr;
  for (int i = 0; i < l.count && !in; ++i)
    if ((uint32_t)l.begin[i].bm == p.tm && (uint32_t)l.begin[i].bn == p.tn && l.begin[i].mode == mode)
      in = l.begin + i;
  if (!in && !rows) return set_error(BST_E_UNSUPPORTED, "no block-scaled kernel with tile %ux%u", p.tm, p.tn);

  BlockGemmArgs a{};
  a.A = A;
  a.B = B;
  a.C = static_cast<uint8_t*>(C);
  a.sa = static_cast<const uint8_t*>(SA);
  a.sb = static_cast<const uint8_t*>(SB);
  a.lda = lda;
  a.ldb = ldb;
  a.ldc = ldc;
  a.ldsa = ldsa;
  a.ldsb = ldsb;
  a.strideB = strideB;
  a.strideSB = strideSB;
  a.group_m = group_m;
  a.G = (uint32_t)G;
  a.M = (uint32_t)M;
  a.N = (uint32_t)N;
  a.K = (uint32_t)K;
  a.nk = (uint32_t)nk;
  a.kslice = (uint32_t)cdiv(nk, p.split);
  a.tiles = (uint32_t)p.tiles;
  a.off = s.off;
  a.dir = s.dir;
  a.remap = s.remap;
  a.grid = (uint32_t)(p.tiles * p.split);
  a.sa_f32 = sa == BST_F32;
  a.sb_f32 = sb == BST_F32;
  a.ckind = (uint32_t)c;
  // a tile's rows of C are stored at 31-bit offsets
  a.cvec = vec_rows(C, ldc, 0, out_bytes(c)) && 256 * ldc * out_bytes(c) < kSpan;
  if (rows) {
    a.grid = (uint32_t)cdiv(N, trans_b ? 16 : 32);
    const dim3 grid(a.grid), block(512);
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, (hipStream_t)stream, a);
      return launched(hipGetLastError(), "block-scaled product");
    };
    const bool exact = mode == MODE_EXACT;
    if (!trans_b) {
      if (M <= 32) return exact ? run(block_rows_n_kernel<1, true>) : run(block_rows_n_kernel<1, false>);
      return exact ? run(block_rows_n_kernel<2, true>) : run(block_rows_n_kernel<2, false>);
    }
    if (M <= 16) return exact ? run(block_rows_kernel<1, true>) : run(block_rows_kernel<1, false>);
    return exact ? run(block_rows_kernel<2, true>) : run(block_rows_kernel<2, false>);
  }
  if (p.split > 1) {
    a.part = static_cast<float*>(ws);
    a.pitch = p.pitch;
  }
  if (!grouped)
    a.mc = make_map_consts((uint32_t)cdiv(M, p.tm), (uint32_t)cdiv(N, p.tn), s.off, s.dir,
                           (uint32_t)p.tiles, a.kslice);
  st = launched(in->launch(a.grid, (hipStream_t)stream, a), "block-scaled product");
  if (st != BST_OK || p.split == 1) return st;
  return reduce(p, 1, M, N, a.part, C, ldc, 0, nullptr, 0, 0, c, stream);
}

bst_status grad(bst_dtype dy, bst_dtype dw, bool grouped, int32_t G, const int32_t* group_m,
                int64_t M, int64_t N, int64_t K, const uint8_t* Q, int64_t ldq, const uint8_t* S,
                int64_t lds, const void* dY, int64_t lddy, const void* add, int64_t ldadd,
                int64_t strideadd, void* dW, int64_t lddw, int64_t stridedw,
                const bst_sched* sched, void* ws, size_t ws_bytes, void* stream) {
  bst_status st = sizes_ok(M, N, K);
  if (st != BST_OK) return st;
  if (!out_bytes(dy)) return set_error(BST_E_UNSUPPORTED, "gradient dtype %d", (int)dy);
  if (!out_bytes(dw)) return set_error(BST_E_UNSUPPORTED, "output dtype %d", (int)dw);
  if (grouped && (st = groups_ok(G, group_m)) != BST_OK) return st;
  Sched s;
  if ((st = read_sched(sched, 0, s)) != BST_OK) return st;
  if (K == 0 || N == 0) return BST_OK;
  const int es = out_bytes(dw);
  if ((st = matrix_ok("dW", dW, lddw, N, es)) != BST_OK) return st;
  if (add && (st = matrix_ok("add", add, ldadd, N, es)) != BST_OK) return st;
  if (grouped && G > 1 && stridedw < (K - 1) * lddw + N)
    return set_error(BST_E_INVAL, "stridedw %lld lets groups of dW overlap (need >= %lld)",
                     (long long)stridedw, (long long)((K - 1) * lddw + N));
  if (grouped && add && strideadd < 0) return set_error(BST_E_INVAL, "negative strideadd");
  if (M > 0) {
    if ((st = codes_ok("Q", Q, ldq, K, 64)) != BST_OK) return st;
    if ((st = scales_ok("S", S, BST_E8M0, lds, cdiv(K, 128))) != BST_OK) return st;
    if ((st = matrix_ok("dY", dY, lddy, N, out_bytes(dy))) != BST_OK) return st;
  }
  Plan p;
  const int kind = dy == BST_BF16 ? DY_BF16 : dy == BST_F16 ? DY_F16 : DY_F32;
  if ((st = plan_grad(grouped ? G : 0, M, N, K, kind + 1, s, p)) != BST_OK) return st;
  if ((st = check_ws(p, ws, ws_bytes)) != BST_OK) return st;
  const BlockGradList l = block_grad_list();
  const BlockGradInstance* in = nullptr;
  for (int i = 0; i < l.count && !in; ++i)
    if ((uint32_t)l.begin[i].bk == p.tm && (uint32_t)l.begin[i].bn == p.tn && l.begin[i].dy == kind)
      in = l.begin + i;
  if (!in) return set_error(BST_E_UNSUPPORTED, "no weight-gradient kernel with tile %ux%u", p.tm, p.tn);

  const int64_t n = grouped ? G : 1;
  BlockGradArgs a{};
  a.Q = Q;
  a.S = S;
  a.dY = static_cast<const uint8_t*>(dY);
  a.add = static_cast<const uint8_t*>(add);
  a.dW = static_cast<uint8_t*>(dW);
  a.ldq = ldq;
  a.lds = lds;
  a.lddy = lddy;
  a.ldadd = ldadd;
  a.lddw = lddw;
  a.strideadd = strideadd;
  a.stridedw = stridedw;
  a.group_m = grouped ? group_m : nullptr;
  a.G = (uint32_t)n;
  a.M = (uint32_t)M;
  a.N = (uint32_t)N;
  a.K = (uint32_t)K;
  a.tiles = (uint32_t)(p.tiles / n);
  a.tiles_all = (uint32_t)p.tiles;
  a.split = p.split;
  a.remap = s.remap;
  a.grid = (uint32_t)(p.tiles * p.split);
  a.dwkind = (uint32_t)dw;
  a.dwvec = vec_rows(dW, lddw, n > 1 ? stridedw : 0, es) &&
            (!add || vec_rows(add, ldadd, n > 1 ? strideadd : 0, es));
  // a stage's 64 rows are loaded at 31-bit offsets
  a.dyvec = vec_rows(dY, lddy, 0, out_bytes(dy)) && 64 * lddy * out_bytes(dy) < kSpan;
  a.mc = make_map_consts((uint32_t)cdiv(K, p.tm), (uint32_t)cdiv(N, p.tn), s.off, s.dir,
                         (uint32_t)p.tiles, 1u);
  if (p.split > 1) {
    a.part = static_cast<float*>(ws);
    a.pitch = p.pitch;
  }
  st = launched(in->launch(a.grid, (hipStream_t)stream, a), "weight gradient");
  if (st != BST_OK || p.split == 1) return st;
  return reduce(p, n, K, N, a.part, dW, lddw, n > 1 ? stridedw : 0, add, ldadd,
                n > 1 ? strideadd : 0, dw, stream);
}

bst_status quant_args(BlockQuantArgs& a, bst_dtype x, int64_t M, int64_t K, int32_t block_rows,
                      int64_t ldx, int64_t ldq, int64_t lds, uint32_t& blocks_rows) {
  bst_status st = sizes_ok(M, 0, K);
  if (st != BST_OK) return st;
  if (!out_bytes(x)) return set_error(BST_E_UNSUPPORTED, "dtype %d", (int)x);
  if (block_rows != 1 && block_rows != 128)
    return set_error(BST_E_UNSUPPORTED, "block_rows %d is neither 1 nor 128", (int)block_rows);
  const int64_t kb = cdiv(K, 128);
  if (ldx < K || ldq < K || lds < kb)
    return set_error(BST_E_INVAL, "leading dimension too small (ldx %lld, ldq %lld, K %lld, lds %lld, "
                     "blocks %lld)", (long long)ldx, (long long)ldq, (long long)K, (long long)lds,
                     (long long)kb);
  if (ldx > kSpan || ldq > kSpan || lds > kSpan)
    return set_error(BST_E_INVAL, "leading dimension above 2^31");
  if (M * kb > kMaxSize) return set_error(BST_E_INVAL, "more than 2^31-1 blocks");
  a.ldx = ldx;
  a.ldq = ldq;
  a.lds = lds;
  a.M = (uint32_t)M;
  a.K = (uint32_t)K;
  a.kb = (uint32_t)kb;
  a.block_rows = (uint32_t)block_rows;
  a.by_kb = make_fastdiv((uint32_t)std::max<int64_t>(kb, 1));
  blocks_rows = (uint32_t)(M * kb);
  return BST_OK;
}

// Workgroups of the row kernels, 16 blocks each and step: enough that the last
// ones to finish do not matter (16384 x 8192 bf16: 79 us with eight per CU, 74
// with 64), fewer when there is less.
uint32_t row_grid(uint32_t blocks) {
  return (uint32_t)std::min<int64_t>(cdiv(blocks, 16), (int64_t)device_cu_count() * 64);
}

}  // namespace

extern "C" {

bst_status bst_quant_block(bst_dtype x, int64_t M, int64_t K, int32_t block_rows, const void* X,
                           int64_t ldx, uint8_t* Q, int64_t ldq, uint8_t* S, int64_t lds,
                           void* stream) {
  BlockQuantArgs a{};
  bst_status st = quant_args(a, x, M, K, block_rows, ldx, ldq, lds, a.blocks);
  if (st != BST_OK) return st;
  const int64_t squares = cdiv(M, 128) * a.kb;
  if (block_rows == 128 && (st = grid_ok(squares, 256)) != BST_OK) return st;
  if (M == 0 || K == 0) return BST_OK;
  if (!X || !Q || !S) return set_error(BST_E_INVAL, "X, Q or S is NULL");
  if (!aligned(X, (uint64_t)out_bytes(x))) return set_error(BST_E_ALIGN, "X is not aligned to its type");
  a.X = static_cast<const uint8_t*>(X);
  a.Q = Q;
  a.S = S;
  a.xvec = vec_rows(X, ldx, 0, out_bytes(x));
  a.qvec = aligned(Q, 8) && ldq % 8 == 0;
  const hipStream_t s = (hipStream_t)stream;
  if (block_rows == 128) {
    const uint32_t grid = (uint32_t)squares;
    if (x == BST_F32)
      hipLaunchKernelGGL((quant_square_kernel<X_F32>), dim3(grid), dim3(256), 0, s, a);
    else if (x == BST_BF16)
      hipLaunchKernelGGL((quant_square_kernel<X_BF16>), dim3(grid), dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((quant_square_kernel<X_F16>), dim3(grid), dim3(256), 0, s, a);
  } else {
    const uint32_t grid = row_grid(a.blocks);
    if (x == BST_F32)
      hipLaunchKernelGGL((quant_rows_kernel<X_F32>), dim3(grid), dim3(256), 0, s, a);
    else if (x == BST_BF16)
      hipLaunchKernelGGL((quant_rows_kernel<X_BF16>), dim3(grid), dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((quant_rows_kernel<X_F16>), dim3(grid), dim3(256), 0, s, a);
  }
  return launched(hipGetLastError(), "quantisation");
}

bst_status bst_dequant_block(bst_dtype x, int64_t M, int64_t K, int32_t block_rows,
                             const uint8_t* Q, int64_t ldq, bst_dtype sk, const void* S, int64_t lds,
                             void* X, int64_t ldx, void* stream) {
  BlockQuantArgs a{};
  bst_status st = quant_args(a, x, M, K, block_rows, ldx, ldq, lds, a.blocks);
  if (st != BST_OK) return st;
  if (!scale_bytes(sk)) return set_error(BST_E_UNSUPPORTED, "scale type %d is neither E8M0 nor F32", (int)sk);
  if (M == 0 || K == 0) return BST_OK;
  if (!X || !Q || !S) return set_error(BST_E_INVAL, "X, Q or S is NULL");
  if (!aligned(X, (uint64_t)out_bytes(x)) || !aligned(S, (uint64_t)scale_bytes(sk)))
    return set_error(BST_E_ALIGN, "X or S is not aligned to its type");
  a.Xo = static_cast<uint8_t*>(X);
  a.Q = const_cast<uint8_t*>(Q);
  a.S = static_cast<uint8_t*>(const_cast<void*>(S));
  a.s_f32 = sk == BST_F32;
  a.xvec = vec_rows(X, ldx, 0, out_bytes(x));
  a.qvec = aligned(Q, 8) && ldq % 8 == 0;
  const uint32_t grid = row_grid(a.blocks);
  const hipStream_t s = (hipStream_t)stream;
  if (x == BST_F32)
    hipLaunchKernelGGL((dequant_kernel<X_F32>), dim3(grid), dim3(256), 0, s, a);
  else if (x == BST_BF16)
    hipLaunchKernelGGL((dequant_kernel<X_BF16>), dim3(grid), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((dequant_kernel<X_F16>), dim3(grid), dim3(256), 0, s, a);
  return launched(hipGetLastError(), "restoring");
}

bst_status bst_gemm_block_scaled(bst_dtype c, int32_t trans_b, int64_t M, int64_t N, int64_t K,
                                 const uint8_t* A, int64_t lda, bst_dtype sa, const void* SA,
                                 int64_t ldsa, const uint8_t* B, int64_t ldb, bst_dtype sb,
                                 const void* SB, int64_t ldsb, void* C, int64_t ldc,
                                 const bst_sched* sched, void* ws, size_t ws_bytes, void* stream) {
  return gemm(c, trans_b, false, 1, nullptr, M, N, K, A, lda, sa, SA, ldsa, B, ldb, 0, sb, SB, ldsb,
              0, C, ldc, sched, ws, ws_bytes, stream);
}

bst_status bst_grouped_gemm_block_scaled(bst_dtype c, int32_t trans_b, int32_t G,
                                         const int32_t* group_m, int64_t total_m, int64_t N,
                                         int64_t K, const uint8_t* A, int64_t lda, bst_dtype sa,
                                         const void* SA, int64_t ldsa, const uint8_t* B, int64_t ldb,
                                         int64_t strideB, bst_dtype sb, const void* SB,
                                         int64_t ldsb, int64_t strideSB, void* C, int64_t ldc,
                                         const bst_sched* sched, void* stream) {
  return gemm(c, trans_b, true, G, group_m, total_m, N, K, A, lda, sa, SA, ldsa, B, ldb, strideB, sb,
              SB, ldsb, strideSB, C, ldc, sched, nullptr, 0, stream);
}

bst_status bst_weight_grad(bst_dtype dy, bst_dtype dw, int64_t M, int64_t N, int64_t K,
                           const uint8_t* Q, int64_t ldq, const uint8_t* S, int64_t lds,
                           const void* dY, int64_t lddy, const void* add, int64_t ldadd, void* dW,
                           int64_t lddw, const bst_sched* sched, void* ws, size_t ws_bytes,
                           void* stream) {
  return grad(dy, dw, false, 1, nullptr, M, N, K, Q, ldq, S, lds, dY, lddy, add, ldadd, 0, dW, lddw,
              0, sched, ws, ws_bytes, stream);
}

bst_status bst_grouped_weight_grad(bst_dtype dy, bst_dtype dw, int32_t G, const int32_t* group_m,
                                   int64_t total_m, int64_t N, int64_t K, const uint8_t* Q,
                                   int64_t ldq, const uint8_t* S, int64_t lds, const void* dY,
                                   int64_t lddy, const void* add, int64_t ldadd, int64_t strideadd,
                                   void* dW, int64_t lddw, int64_t stridedw,
                                   const bst_sched* sched, void* ws, size_t ws_bytes,
                                   void* stream) {
  return grad(dy, dw, true, G, group_m, total_m, N, K, Q, ldq, S, lds, dY, lddy, add, ldadd,
              strideadd, dW, lddw, stridedw, sched, ws, ws_bytes, stream);
}

size_t bst_block_workspace_bytes(int kind, int64_t count, int64_t M, int64_t N, int64_t K,
                                 const bst_sched* sched) {
  Sched s;
  Plan p;
  if (kind < 0 || kind > 3) {
    set_error(BST_E_INVAL, "workspace kind %d not in {0, 1, 2, 3}", kind);
    return 0;
  }
  if (sizes_ok(M, N, K) != BST_OK || read_sched(sched, kind == 0 || kind == 3 ? 128 : 0, s) != BST_OK)
    return 0;
  if (kind == 2 && (count < 1 || count > kMaxGroups)) {
    set_error(BST_E_INVAL, "group count %lld outside [1, %d]", (long long)count, kMaxGroups);
    return 0;
  }
  if ((kind == 0 || kind == 3) && takes_rows(kind == 3, M, N, K, s)) return 0;
  // the types, which may change the tile or the split, are not known here:
  // enough for any
  if (kind == 1 || kind == 2) {
    size_t most = 0;
    for (int parts = 1; parts <= 3; ++parts) {
      Plan q;
      if (plan_grad(kind == 2 ? count : 0, M, N, K, parts, s, q) == BST_OK) most = std::max(most, q.ws);
    }
    return most;
  }
  Plan q;
  const bst_status other = plan_gemm(0, M, N, K, true, s, q);
  const bst_status st = plan_gemm(0, M, N, K, false, s, p);
  return std::max(st == BST_OK ? p.ws : 0, other == BST_OK ? q.ws : 0);
}

}  // extern "C"
