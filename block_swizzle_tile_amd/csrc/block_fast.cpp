// block_fast.cpp -- the short way from Python to the block-scaled operators.
//
// A call with new outputs, no schedule and no workspace of the caller's, on
// tensors of the current device that need no special treatment, goes through
// here: the same checks as block.py, the allocation of the outputs and the
// workspace from torch's allocator, and the call of the C ABI, in one C
// function (quantising one row 8.7 us of host time through ctypes, 5 here).
// Whatever it does not take, or the C ABI refuses, it answers with None, and
// block.py's own path runs, which states what is wrong.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/hip/HIPFunctions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "bst_block.h"

namespace {

decltype(&bst_quant_block) f_quant = nullptr;
decltype(&bst_dequant_block) f_dequant = nullptr;
decltype(&bst_gemm_block_scaled) f_gemm = nullptr;
decltype(&bst_grouped_gemm_block_scaled) f_grouped = nullptr;
decltype(&bst_weight_grad) f_grad = nullptr;
decltype(&bst_grouped_weight_grad) f_ggrad = nullptr;
decltype(&bst_block_workspace_bytes) f_ws = nullptr;

constexpr at::ScalarType kCodes = at::kFloat8_e4m3fn;

struct NotTaken {};  // thrown by the checks, caught at each entry

void need(bool ok) {
  if (!ok) throw NotTaken{};
}

const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

bst_dtype out_type(at::ScalarType t) {
  if (t == at::kBFloat16) return BST_BF16;
  if (t == at::kHalf) return BST_F16;
  need(t == at::kFloat);
  return BST_F32;
}

bst_dtype scale_type(const at::Tensor& t) {
  const at::ScalarType s = t.scalar_type();
  if (s == at::kFloat) return BST_F32;
  need(s == at::kByte || s == at::kFloat8_e8m0fnu);
  return BST_E8M0;
}

// The type that a dtype argument names, or `other` for None.
at::ScalarType dtype_or(PyObject* o, at::ScalarType other) {
  if (o == Py_None) return other;
  need(THPDtype_Check(o));
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
int64_t blocks(int64_t n) { return (n + 127) / 128; }

// Pitch of a matrix of rows x cols (of the last two dimensions): as block.py's.
int64_t pitch(const at::Tensor& t, int64_t rows, int64_t cols, int64_t pad = 1) {
  const int64_t d = t.dim();
  need(d >= 2 && t.size(d - 2) == rows && t.size(d - 1) == cols);
  need(cols <= 1 || t.stride(d - 1) == 1);
  return rows > 1 ? t.stride(d - 2) : up(cols, pad);
}

// All on the current GPU, plain strided tensors.
void here(std::initializer_list<const at::Tensor*> ts) {
  const int d = c10::hip::current_device();
  for (const at::Tensor* t : ts)
    need(t->is_cuda() && t->get_device() == d && t->layout() == at::kStrided);
}

void* stream() {
  return c10::hip::getCurrentHIPStreamMasqueradingAsCUDA().stream();
}

template <typename T = void>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

at::Tensor make(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
  return at::empty(shape, like.options().dtype(type).requires_grad(false));
}

PyObject* none() { Py_RETURN_NONE; }

// Runs an entry; anything that it does not take or that fails becomes None.
template <typename F>
PyObject* entry(F&& f) {
  try {
    return f();
  } catch (const NotTaken&) {
  } catch (const std::exception&) {
  }
  PyErr_Clear();
  return none();
}

// quant(X, block_rows) -> (Q, scale)
PyObject* quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry([&]() -> PyObject* {
    need(n == 2 && PyLong_Check(a[1]));
    const at::Tensor& x = tensor(a[0]);
    const long br = PyLong_AsLong(a[1]);
    need(br == 1 || br == 128);
    here({&x});
    need(x.dim() == 2);
    const int64_t M = x.size(0), K = x.size(1), kb = blocks(K), ldq = up(K, 16);
    const int64_t ldx = pitch(x, M, K);
    const bst_dtype kind = out_type(x.scalar_type());
    at::Tensor q = make(x, {M, ldq}, kCodes);
    at::Tensor s = make(x, {br == 1 ? M : blocks(M), kb}, at::kByte);
    need(f_quant(kind, M, K, (int32_t)br, ptr(x), ldx, ptr<uint8_t>(q), ldq, ptr<uint8_t>(s), kb,
                 stream()) == BST_OK);
    if (ldq != K) q = q.narrow(1, 0, K);
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(s)));
  });
}

// dequant(Q, scale, dtype, block_rows) -> X
PyObject* dequant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry([&]() -> PyObject* {
    need(n == 4 && PyLong_Check(a[3]));
    const at::Tensor &q = tensor(a[0]), &s = tensor(a[1]);
    const at::ScalarType type = dtype_or(a[2], at::kBFloat16);
    const long br = PyLong_AsLong(a[3]);
    need(br == 1 || br == 128);
    here({&q, &s});
    need(q.dim() == 2 && s.dim() == 2 && q.scalar_type() == kCodes);
    const int64_t M = q.size(0), K = q.size(1);
    const int64_t ldq = pitch(q, M, K), lds = pitch(s, br == 1 ? M : blocks(M), blocks(K));
    const bst_dtype kind = out_type(type), sk = scale_type(s);
    at::Tensor x = make(q, {M, K}, type);
    need(f_dequant(kind, M, K, (int32_t)br, ptr<uint8_t>(q), ldq, sk, ptr(s), lds, ptr(x), K,
                   stream()) == BST_OK);
    return THPVariable_Wrap(std::move(x));
  });
}

// What the two products take of their operands.
struct Product {
  int64_t M, N, K, lda, ldb, ldsa, ldsb;
  bst_dtype ka, kb;
  Product(const at::Tensor& A, const at::Tensor& B, const at::Tensor& sa, const at::Tensor& sb,
          bool tb, int64_t G) {
    const int64_t d = G ? 3 : 2;
    need(A.scalar_type() == kCodes && B.scalar_type() == kCodes);
    need(A.dim() == 2 && B.dim() == d && sa.dim() == 2 && sb.dim() == d);
    need(!G || (B.size(0) == G && sb.size(0) == G));
    M = A.size(0);
    K = A.size(1);
    N = B.size(tb ? d - 2 : d - 1);
    lda = pitch(A, M, K, 16);
    ldb = tb ? pitch(B, N, K, 16) : pitch(B, K, N, 16);
    ldsa = pitch(sa, M, blocks(K));
    ldsb = tb ? pitch(sb, blocks(N), blocks(K)) : pitch(sb, blocks(K), blocks(N));
    ka = scale_type(sa);
    kb = scale_type(sb);
  }
};

int64_t group_count(const at::Tensor& gm) {
  need(gm.scalar_type() == at::kInt && gm.dim() == 1 && gm.is_contiguous() && gm.size(0) > 0);
  return gm.size(0);
}

// gemm(A, B, scale_a, scale_b, trans_b, dtype) -> C
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry([&]() -> PyObject* {
    need(n == 6);
    const at::Tensor &A = tensor(a[0]), &B = tensor(a[1]), &sa = tensor(a[2]), &sb = tensor(a[3]);
    const bool tb = a[4] == Py_True;
    const at::ScalarType type = dtype_or(a[5], at::kBFloat16);
    here({&A, &B, &sa, &sb});
    const Product p(A, B, sa, sb, tb, 0);
    const bst_dtype kind = out_type(type);
    at::Tensor C = make(A, {p.M, p.N}, type), ws;
    const size_t need_ws = f_ws(tb ? 3 : 0, 1, p.M, p.N, p.K, nullptr);
    if (need_ws) ws = make(A, {(int64_t)need_ws}, at::kByte);
    need(f_gemm(kind, tb, p.M, p.N, p.K, ptr<uint8_t>(A), p.lda, p.ka, ptr(sa), p.ldsa,
                ptr<uint8_t>(B), p.ldb, p.kb, ptr(sb), p.ldsb, ptr(C), p.N, nullptr,
                need_ws ? ptr(ws) : nullptr, need_ws, stream()) == BST_OK);
    return THPVariable_Wrap(std::move(C));
  });
}

// grouped(A, B, group_m, scale_a, scale_b, trans_b, dtype) -> C
PyObject* grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry([&]() -> PyObject* {
    need(n == 7);
    const at::Tensor &A = tensor(a[0]), &B = tensor(a[1]), &gm = tensor(a[2]), &sa = tensor(a[3]),
                     &sb = tensor(a[4]);
    const bool tb = a[5] == Py_True;
    const at::ScalarType type = dtype_or(a[6], at::kBFloat16);
    here({&A, &B, &gm, &sa, &sb});
    const int64_t G = group_count(gm);
    const Product p(A, B, sa, sb, tb, G);
    const bst_dtype kind = out_type(type);
    at::Tensor C = make(A, {p.M, p.N}, type);
    need(f_grouped(kind, tb, (int32_t)G, ptr<int32_t>(gm), p.M, p.N, p.K, ptr<uint8_t>(A), p.lda,
                   p.ka, ptr(sa), p.ldsa, ptr<uint8_t>(B), p.ldb, G > 1 ? B.stride(0) : 0, p.kb,
                   ptr(sb), p.ldsb, G > 1 ? sb.stride(0) : 0, ptr(C), p.N, nullptr,
                   stream()) == BST_OK);
    return THPVariable_Wrap(std::move(C));
  });
}

// grad(Q, scale, dY, group_m or None, add or None, dtype or None) -> dW
PyObject* grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry([&]() -> PyObject* {
    need(n == 6);
    const at::Tensor &q = tensor(a[0]), &s = tensor(a[1]), &dy = tensor(a[2]);
    const at::Tensor* gm = a[3] == Py_None ? nullptr : &tensor(a[3]);
    const at::Tensor* add = a[4] == Py_None ? nullptr : &tensor(a[4]);
    const at::ScalarType type = dtype_or(a[5], add ? add->scalar_type() : at::kFloat);
    here({&q, &s, &dy});
    if (gm) here({gm});
    if (add) here({add});
    need(q.dim() == 2 && s.dim() == 2 && dy.dim() == 2 && q.scalar_type() == kCodes);
    need(scale_type(s) == BST_E8M0);
    const int64_t M = q.size(0), K = q.size(1), N = dy.size(1), G = gm ? group_count(*gm) : 1;
    const int64_t ldq = pitch(q, M, K, 16), lds = pitch(s, M, blocks(K)), ldy = pitch(dy, M, N);
    int64_t lda = 0, stride = 0;
    if (add) {
      need(add->scalar_type() == type && add->dim() == (gm ? 3 : 2) && (!gm || add->size(0) == G));
      lda = pitch(*add, K, N);
      stride = G > 1 ? add->stride(0) : 0;
    }
    const bst_dtype kind = out_type(type), dk = out_type(dy.scalar_type());
    at::Tensor w = gm ? make(q, {G, K, N}, type) : make(q, {K, N}, type), ws;
    const size_t need_ws = f_ws(gm ? 2 : 1, G, M, N, K, nullptr);
    if (need_ws) ws = make(q, {(int64_t)need_ws}, at::kByte);
    void* const wp = need_ws ? ptr(ws) : nullptr;
    const void* const ap = add ? ptr(*add) : nullptr;
    const bst_status st =
        gm ? f_ggrad(dk, kind, (int32_t)G, ptr<int32_t>(*gm), M, N, K, ptr<uint8_t>(q), ldq,
                     ptr<uint8_t>(s), lds, ptr(dy), ldy, ap, lda, stride, ptr(w), N,
                     G > 1 ? K * N : 0, nullptr, wp, need_ws, stream())
           : f_grad(dk, kind, M, N, K, ptr<uint8_t>(q), ldq, ptr<uint8_t>(s), lds, ptr(dy), ldy, ap,
                    lda, ptr(w), N, nullptr, wp, need_ws, stream());
    need(st == BST_OK);
    return THPVariable_Wrap(std::move(w));
  });
}

// bind(addresses of the seven C functions, in the order below)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
    return nullptr;
  }
  void* p[7];
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a NULL address");
      return nullptr;
    }
  }
  f_quant = reinterpret_cast<decltype(f_quant)>(p[0]);
  f_dequant = reinterpret_cast<decltype(f_dequant)>(p[1]);
  f_gemm = reinterpret_cast<decltype(f_gemm)>(p[2]);
  f_grouped = reinterpret_cast<decltype(f_grouped)>(p[3]);
  f_grad = reinterpret_cast<decltype(f_grad)>(p[4]);
  f_ggrad = reinterpret_cast<decltype(f_ggrad)>(p[5]);
  f_ws = reinterpret_cast<decltype(f_ws)>(p[6]);
  return none();
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant)), METH_FASTCALL, nullptr},
    {"dequant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(dequant)), METH_FASTCALL, nullptr},
    {"gemm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gemm)), METH_FASTCALL, nullptr},
    {"grouped", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grouped)), METH_FASTCALL, nullptr},
    {"grad", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grad)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_block_fast", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_fast() { return PyModule_Create(&module_def); }
