// fast.hpp -- what the short ways from Python to the operators share
// (block_fast.cpp, more_fast.cpp): checks that answer "not taken", the outputs'
// allocation, the current stream.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <ATen/record_function.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/hip/HIPFunctions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "bst_block.h"

namespace fast {

struct NotTaken {};  // thrown by the checks, caught at each entry

inline void need(bool ok) {
  if (!ok) throw NotTaken{};
}

inline const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

inline bst_dtype out_type(at::ScalarType t) {
  if (t == at::kBFloat16) return BST_BF16;
  if (t == at::kHalf) return BST_F16;
  need(t == at::kFloat);
  return BST_F32;
}

inline bst_dtype scale_type(const at::Tensor& t) {
  const at::ScalarType s = t.scalar_type();
  if (s == at::kFloat) return BST_F32;
  need(s == at::kByte || s == at::kFloat8_e8m0fnu);
  return BST_E8M0;
}

// The type that a dtype argument names, or `other` for None.
inline at::ScalarType dtype_or(PyObject* o, at::ScalarType other) {
  if (o == Py_None) return other;
  need(THPDtype_Check(o));
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

inline int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// Pitch of a matrix of rows x cols (of the last two dimensions): as block.py's.
inline int64_t pitch(const at::Tensor& t, int64_t rows, int64_t cols, int64_t pad = 1) {
  const int64_t d = t.dim();
  need(d >= 2 && t.size(d - 2) == rows && t.size(d - 1) == cols);
  need(cols <= 1 || t.stride(d - 1) == 1);
  return rows > 1 ? t.stride(d - 2) : up(cols, pad);
}

// All on the current GPU, plain strided tensors.
inline void here(std::initializer_list<const at::Tensor*> ts) {
  const int d = c10::hip::current_device();
  for (const at::Tensor* t : ts)
    need(t->is_cuda() && t->get_device() == d && t->layout() == at::kStrided);
}

inline void* stream() {
  return c10::hip::getCurrentHIPStreamMasqueradingAsCUDA().stream();
}

template <typename T = void>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// Whether anything listens to torch's dispatcher: a mode, a transform or a tracer (keys
// of this thread beside those that are always there), or a profiler.
inline bool heard() {
  return !(c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty() ||
         at::hasCallbacks();
}

// An empty tensor on the inputs' device, without the dispatcher's way to it (half a
// microsecond), unless torch fills new tensors or something is there to see them.
inline at::Tensor make(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
  if (at::globalContext().deterministicAlgorithms() || heard())
    return at::empty(shape, like.options().dtype(type).requires_grad(false));
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

inline PyObject* none() { Py_RETURN_NONE; }

// Runs an entry; anything that it does not take or that fails becomes None.
template <typename F>
inline PyObject* entry(F&& f) {
  try {
    return f();
  } catch (const NotTaken&) {
  } catch (const std::exception&) {
  }
  PyErr_Clear();
  return none();
}

// The methods of more_fast.cpp, ended by an entry without a name.
extern PyMethodDef more_methods[];

}  // namespace fast
