// moe.hip -- host side of the operators declared in include/bst_moe.h:
// argument checks (before any HIP call), the choice of kernel, the launches.
#include "bst_host.hpp"
#include "bst_moe.hpp"

using namespace bst;
using namespace bst::host;

namespace {

// Choices that one launch takes, whose workgroups, one for each expert, read all of
// them (128 experts, in one launch and in two: 8192 choices 3.8 us and 9.4, 32768
// 7.2 and 10.6, 65536 11.8 and 9.0).
bool sorts_at_once(int64_t n, int32_t G) { return n <= 32768 && n * G <= 1 << 23; }

struct SortPlan {
  uint32_t chunk = 0, chunks = 0, pitch = 0;
  size_t ws = 0;
};

// At most 512 chunks: each chunk's workgroup reads the counts of all.
SortPlan plan_sort(int64_t n, int32_t G) {
  SortPlan p;
  if (sorts_at_once(n, G)) return p;
  p.chunk = (uint32_t)(cdiv(std::max<int64_t>(cdiv(n, 512), 1024), 256) * 256);
  p.chunks = (uint32_t)cdiv(n, p.chunk);
  p.pitch = (uint32_t)(cdiv(G, 4) * 4);
  p.ws = (size_t)p.chunks * p.pitch * 4;
  return p;
}

bst_status experts_ok(int64_t n, int32_t G) {
  if (G < 1 || G > kMaxGroups)
    return set_error(BST_E_INVAL, "expert count %d outside [1, %d]", (int)G, kMaxGroups);
  if (n < 0) return set_error(BST_E_INVAL, "negative size");
  if (n > kMaxSize) return set_error(BST_E_INVAL, "more than 2^31-1 choices");
  return BST_OK;
}

bst_status choices_ok(int64_t T, int32_t k, int64_t rows) {
  if (T < 0 || k < 0 || rows < 0) return set_error(BST_E_INVAL, "negative size");
  if (T > kMaxSize || rows > kMaxSize) return set_error(BST_E_INVAL, "size above 2^31-1");
  if (k > 0 && T > kMaxSize / k) return set_error(BST_E_INVAL, "more than 2^31-1 choices");
  return BST_OK;
}

bst_status row_of_ok(const int32_t* row_of) {
  if (!row_of) return set_error(BST_E_INVAL, "row_of is NULL");
  if (!aligned(row_of, 4)) return set_error(BST_E_ALIGN, "row_of is not 4-byte aligned");
  return BST_OK;
}

// Workgroups of 256 threads, one thread each item; the kernels count items in 32 bits.
bst_status threads_ok(int64_t items) {
  if (items > 0xffffffffLL - 255)
    return set_error(BST_E_UNSUPPORTED, "%lld pieces of rows are more threads than one launch holds",
                     (long long)items);
  return BST_OK;
}

bst_status moe_rows(MoeRows& m, const char* what, const char* dst, int64_t T, int64_t bytes, const void* X,
                    int64_t ldx, void* R, int64_t ldr) {
  if (ldx < bytes || ldr < bytes)
    return set_error(BST_E_INVAL, "%s or %s: pitch below the %lld bytes of a row", what, dst,
                     (long long)bytes);
  if (ldx > 4 * kSpan || ldr > 4 * kSpan)
    return set_error(BST_E_INVAL, "%s or %s: pitch above 2^33 bytes", what, dst);
  m.x = static_cast<const uint8_t*>(X);
  m.r = static_cast<uint8_t*>(R);
  m.ldx = ldx;
  m.ldr = ldr;
  m.bytes = (uint32_t)bytes;
  m.pieces = (uint32_t)cdiv(bytes, 16);
  m.by_pieces = make_fastdiv(m.pieces);
  return threads_ok(T * (int64_t)m.pieces);
}

}  // namespace

extern "C" {

size_t bst_moe_workspace_bytes(int64_t n, int32_t G) {
  if (experts_ok(n, G) != BST_OK) return 0;
  return plan_sort(n, G).ws;
}

bst_status bst_moe_sort(int32_t id_bytes, int64_t n, const void* expert, int32_t first, int32_t G,
                        int32_t* row_of, int32_t* group_m, void* ws, size_t ws_bytes, void* stream) {
  bst_status st = experts_ok(n, G);
  if (st != BST_OK) return st;
  if (id_bytes != 4 && id_bytes != 8)
    return set_error(BST_E_UNSUPPORTED, "expert ids of %d bytes", (int)id_bytes);
  if (first < 0 || first > kMaxSize - G)
    return set_error(BST_E_INVAL, "experts %d .. %lld are outside [0, 2^31-1)", (int)first, (long long)first + G - 1);
  if (!group_m) return set_error(BST_E_INVAL, "group sizes are NULL");
  if (!aligned(group_m, 4)) return set_error(BST_E_ALIGN, "group sizes are not 4-byte aligned");
  if (n > 0) {
    if (!expert) return set_error(BST_E_INVAL, "expert is NULL");
    if (!aligned(expert, (uint64_t)id_bytes)) return set_error(BST_E_ALIGN, "expert is not aligned to its type");
    if ((st = row_of_ok(row_of)) != BST_OK) return st;
  }
  const SortPlan p = plan_sort(n, G);
  if (p.ws) {
    if (!ws || ws_bytes < p.ws)
      return set_error(BST_E_WORKSPACE, "%lld choices of %d experts need %zu workspace bytes (got %zu)",
                       (long long)n, (int)G, p.ws, ws ? ws_bytes : (size_t)0);
    if (!aligned(ws, 16)) return set_error(BST_E_ALIGN, "workspace not 16-byte aligned");
  }
  MoeSortArgs a{};
  a.expert = expert;
  a.row_of = row_of;
  a.group_m = group_m;
  a.counts = static_cast<uint32_t*>(ws);
  a.first = first;
  a.n = (uint32_t)n;
  a.G = (uint32_t)G;
  a.pitch = p.pitch;
  a.chunk = p.chunk;
  a.chunks = p.chunks;
  const hipStream_t s = (hipStream_t)stream;
  const dim3 block(256);
  if (!p.ws) {
    const dim3 grid(a.G);
    if (n <= 2048) {
      if (id_bytes == 4) hipLaunchKernelGGL((moe_sort_one<int32_t, 4>), grid, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((moe_sort_one<int64_t, 4>), grid, dim3(256), 0, s, a);
    } else {
      if (id_bytes == 4) hipLaunchKernelGGL((moe_sort_one<int32_t, 16>), grid, dim3(1024), 0, s, a);
      else hipLaunchKernelGGL((moe_sort_one<int64_t, 16>), grid, dim3(1024), 0, s, a);
    }
    return launched(hipGetLastError(), "expert sort");
  }
  if (id_bytes == 4) hipLaunchKernelGGL((moe_count<int32_t>), dim3(a.chunks), block, 0, s, a);
  else hipLaunchKernelGGL((moe_count<int64_t>), dim3(a.chunks), block, 0, s, a);
  if ((st = launched(hipGetLastError(), "expert count")) != BST_OK) return st;
  if (id_bytes == 4) hipLaunchKernelGGL((moe_place<int32_t>), dim3(a.chunks), block, 0, s, a);
  else hipLaunchKernelGGL((moe_place<int64_t>), dim3(a.chunks), block, 0, s, a);
  return launched(hipGetLastError(), "expert sort");
}

bst_status bst_moe_gather(int64_t T, int32_t k, int64_t row_bytes, const void* X, int64_t ldx,
                          const int32_t* row_of, int64_t rows, void* R, int64_t ldr, int64_t scale_bytes,
                          const void* S, int64_t lds, void* RS, int64_t ldrs, void* stream) {
  bst_status st = choices_ok(T, k, rows);
  if (st != BST_OK) return st;
  if (row_bytes < 0 || scale_bytes < 0) return set_error(BST_E_INVAL, "negative size");
  if (row_bytes > 4 * kMaxSize || scale_bytes > 4 * kMaxSize)
    return set_error(BST_E_INVAL, "rows of more than 2^33 bytes");
  if (!S) scale_bytes = 0;
  if (T == 0 || k == 0 || rows == 0 || (row_bytes == 0 && scale_bytes == 0)) return BST_OK;
  if ((row_bytes && (!X || !R)) || (scale_bytes && !RS)) return set_error(BST_E_INVAL, "a matrix is NULL");
  if ((st = row_of_ok(row_of)) != BST_OK) return st;
  if (row_bytes > 0xfffffff0LL || scale_bytes > 0xfffffff0LL)
    return set_error(BST_E_UNSUPPORTED, "rows of more than 2^32 bytes");
  MoeGatherArgs a{};
  if ((st = moe_rows(a.m[0], "X", "R", T, row_bytes, X, ldx, R, ldr)) != BST_OK) return st;
  if (scale_bytes && (st = moe_rows(a.m[1], "S", "RS", T, scale_bytes, S, lds, RS, ldrs)) != BST_OK) return st;
  const int64_t items = T * ((int64_t)a.m[0].pieces + a.m[1].pieces);
  if ((st = threads_ok(items)) != BST_OK) return st;
  a.row_of = row_of;
  a.T = (uint32_t)T;
  a.k = (uint32_t)k;
  a.rows = (uint32_t)rows;
  const dim3 grid((uint32_t)cdiv(items, 256)), block(256);
  if (is_far(T * k, row_bytes)) hipLaunchKernelGGL(moe_gather_kernel<true>, grid, block, 0, (hipStream_t)stream, a);
  else hipLaunchKernelGGL(moe_gather_kernel<false>, grid, block, 0, (hipStream_t)stream, a);
  return launched(hipGetLastError(), "gather");
}

bst_status bst_moe_combine(bst_dtype r, bst_dtype y, int64_t T, int32_t k, int64_t H, const void* R,
                           int64_t ldr, int64_t rows, const int32_t* row_of, bst_dtype w,
                           const void* weights, const void* add, int64_t ldadd, void* Y, int64_t ldy,
                           void* stream) {
  bst_status st = choices_ok(T, k, rows);
  if (st != BST_OK) return st;
  if ((st = sizes_ok(T, 0, H)) != BST_OK) return st;
  const int er = out_bytes(r), ey = out_bytes(y), ew = out_bytes(w);
  if (!er) return set_error(BST_E_UNSUPPORTED, "row dtype %d", (int)r);
  if (!ey) return set_error(BST_E_UNSUPPORTED, "output dtype %d", (int)y);
  if (weights && !ew) return set_error(BST_E_UNSUPPORTED, "weight dtype %d", (int)w);
  if (T == 0 || H == 0) return BST_OK;
  if ((st = matrix_ok("Y", Y, ldy, H, ey)) != BST_OK) return st;
  if (add && (st = matrix_ok("add", add, ldadd, H, ey)) != BST_OK) return st;
  const bool any = k > 0 && rows > 0;
  if (any) {
    if ((st = matrix_ok("R", R, ldr, H, er)) != BST_OK) return st;
    if ((st = row_of_ok(row_of)) != BST_OK) return st;
    if (weights && !aligned(weights, (uint64_t)ew))
      return set_error(BST_E_ALIGN, "weights are not aligned to their type");
  }
  MoeCombineArgs a{};
  a.pieces = (uint32_t)cdiv(H, r == BST_F32 ? kCols<X_F32> : kCols<X_BF16>);
  if ((st = threads_ok(T * (int64_t)a.pieces)) != BST_OK) return st;
  a.R = static_cast<const uint8_t*>(R);
  a.w = static_cast<const uint8_t*>(weights);
  a.add = static_cast<const uint8_t*>(add);
  a.Y = static_cast<uint8_t*>(Y);
  a.row_of = row_of;
  a.ldr = ldr * er;
  a.ldadd = ldadd * ey;
  a.ldy = ldy * ey;
  a.T = (uint32_t)T;
  a.k = any ? (uint32_t)k : 0u;
  a.H = (uint32_t)H;
  a.rows = (uint32_t)rows;
  a.wkind = (uint32_t)w;
  a.ykind = (uint32_t)y;
  a.by_pieces = make_fastdiv(a.pieces);
  const dim3 grid((uint32_t)cdiv(T * (int64_t)a.pieces, 256)), block(256);
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, (hipStream_t)stream, a);
    return launched(hipGetLastError(), "combine");
  };
  const bool far = is_far(T * k, H * er);
  auto pick = [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    return far ? run(moe_combine_kernel<KIND, true>) : run(moe_combine_kernel<KIND, false>);
  };
  if (r == BST_F32) return pick(std::integral_constant<int, X_F32>{});
  if (r == BST_BF16) return pick(std::integral_constant<int, X_BF16>{});
  return pick(std::integral_constant<int, X_F16>{});
}

bst_status bst_moe_combine_grad(bst_dtype r, int64_t T, int32_t k, int64_t H, const void* dY, int64_t lddy,
                                const void* R, int64_t ldr, int64_t rows, const int32_t* row_of,
                                bst_dtype w, const void* weights, void* dR, int64_t lddr, void* dweights,
                                void* stream) {
  bst_status st = choices_ok(T, k, rows);
  if (st != BST_OK) return st;
  if ((st = sizes_ok(T, 0, H)) != BST_OK) return st;
  const int er = out_bytes(r), ew = out_bytes(w);
  if (!er) return set_error(BST_E_UNSUPPORTED, "row dtype %d", (int)r);
  if (!ew) return set_error(BST_E_UNSUPPORTED, "weight dtype %d", (int)w);
  if (T == 0 || k == 0 || (!dR && !dweights)) return BST_OK;
  if (!weights) return set_error(BST_E_INVAL, "weights are NULL");
  if (!aligned(weights, (uint64_t)ew) || !aligned(dweights, (uint64_t)ew))
    return set_error(BST_E_ALIGN, "weights or dweights are not aligned to their type");
  if ((st = row_of_ok(row_of)) != BST_OK) return st;
  const bool any = H > 0 && rows > 0;
  if (any) {
    if ((st = matrix_ok("dY", dY, lddy, H, er)) != BST_OK) return st;
    if (dweights && (st = matrix_ok("R", R, ldr, H, er)) != BST_OK) return st;
    if (dR && (st = matrix_ok("dR", dR, lddr, H, er)) != BST_OK) return st;
  }
  // Four waves a token where its row keeps them busy, or where there are too few
  // tokens to fill the chip with a wave each (8192 x 4 rows of 4096 bf16: 147 us with
  // one wave, 136 with four; 4000 x 8 rows of 1024: 34, 55; 500 x 4 rows of 1000 fp32
  // 9.4, 6.1).  Of few tokens every four choices are a task of their own (700 x 8 rows
  // of 2048 bf16: 10.7 us without, 9.6 with it, 1000 x 8 rows of 600 10.4, 7.7, of 2048
  // 13.5, 14.9), of sixteen waves where those leave CUs without work (20 x 6 rows of
  // 7168 fp16: 11.9 us with a workgroup of four waves a token, 5.8; past the caches 256 x 4
  // rows of 8192 bf16 18.7 us with four, 11.1 with sixteen, 64 x 8 rows of 8192 fp32 34.2,
  // 15.8).
  const int64_t cus = device_cu_count(), lanes = cdiv(H * er, 16);  // that a row keeps busy
  const int64_t parts = T < cus * 4 && lanes > 64 ? cdiv(k, 4) : 1;
  const int waves = lanes > 256 && T * parts <= cus ? 16 : lanes >= 256 || (lanes > 64 && T < cus * 2) ? 4 : 1;
  const int64_t groups = waves > 1 ? T * parts : cdiv(T * parts, 4);
  if ((st = grid_ok(groups, 64 * std::max(waves, 4))) != BST_OK) return st;
  MoeGradArgs a{};
  a.dY = static_cast<const uint8_t*>(dY);
  a.R = static_cast<const uint8_t*>(R);
  a.w = static_cast<const uint8_t*>(weights);
  a.dR = static_cast<uint8_t*>(dR);
  a.dw = static_cast<uint8_t*>(dweights);
  a.row_of = row_of;
  a.lddy = lddy * er;
  a.ldr = ldr * er;
  a.lddr = lddr * er;
  a.T = (uint32_t)T;
  a.k = (uint32_t)k;
  a.H = (uint32_t)H;
  a.rows = any ? (uint32_t)rows : 0u;
  a.wkind = (uint32_t)w;
  a.parts = (uint32_t)parts;
  a.by_parts = make_fastdiv(a.parts);
  const bool far = is_far(T * k, H * er);
  // a launch's threads are those of its kernel
  auto run = [&](auto kind, auto wpt) {
    constexpr int KIND = decltype(kind)::value, WPT = decltype(wpt)::value;
    const dim3 grid((uint32_t)groups), block(kGradThreads<WPT>);
    if (far) hipLaunchKernelGGL((moe_combine_grad_kernel<KIND, WPT, true>), grid, block, 0, (hipStream_t)stream, a);
    else hipLaunchKernelGGL((moe_combine_grad_kernel<KIND, WPT, false>), grid, block, 0, (hipStream_t)stream, a);
    return launched(hipGetLastError(), "combine gradient");
  };
  auto pick = [&](auto kind) {
    if (waves == 16) return run(kind, std::integral_constant<int, 16>{});
    if (waves == 4) return run(kind, std::integral_constant<int, 4>{});
    return run(kind, std::integral_constant<int, 1>{});
  };
  if (r == BST_F32) return pick(std::integral_constant<int, X_F32>{});
  if (r == BST_BF16) return pick(std::integral_constant<int, X_BF16>{});
  return pick(std::integral_constant<int, X_F16>{});
}

}  // extern "C"
