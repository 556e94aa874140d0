// torch_calls.h -- what the marshalling of all operators shares: the bound entry
// points, checks of tensors, streams and the versions of what a call writes.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/util/SmallVector.h>

#include <mutex>
#include <vector>

#include "../../include/gdn_prefill.h"

namespace calls {

using at::Tensor;

// ------------------------------------------------------------------- library

struct Bound {
  size_t (*rec_workspace)(const gdn_recurrence_params *, int32_t) = nullptr;
  int (*rec_forward)(const gdn_recurrence_params *, void *) = nullptr;
  int (*rec_backward)(const gdn_recurrence_params *, void *) = nullptr;
  int (*rec_decode)(const gdn_recurrence_params *, void *) = nullptr;
  int (*pool_copy)(const gdn_pool_params *, void *) = nullptr;
  int (*pool_reset)(const gdn_pool_params *, void *) = nullptr;
  int (*pool_compact)(const gdn_pool_params *, void *, int32_t *, int32_t *, void *) = nullptr;
  int (*pool_validate)(const gdn_pool_params *, int32_t) = nullptr;
  size_t (*conv_workspace)(const gdn_convolution_params *, int32_t) = nullptr;
  int (*conv_forward)(const gdn_convolution_params *, void *) = nullptr;
  int (*conv_backward)(const gdn_convolution_params *, void *) = nullptr;
  int (*conv_decode)(const gdn_convolution_params *, void *) = nullptr;
  int64_t (*scan_chunk)(const gdn_scan_params *) = nullptr;
  size_t (*scan_workspace)(const gdn_scan_params *, int32_t) = nullptr;
  int (*scan_forward)(const gdn_scan_params *, void *) = nullptr;
  int (*scan_backward)(const gdn_scan_params *, void *) = nullptr;
  int (*scan_decode)(const gdn_scan_params *, void *) = nullptr;
  size_t (*beam_workspace)(const gdn_beam_params *) = nullptr;
  int (*beam_select)(const gdn_beam_params *, void *) = nullptr;
  int (*pool_reorder)(const gdn_reorder_params *, void *) = nullptr;
  PyObject *raise = nullptr;      // raise(code): the exception of an error code
  PyObject *stream = nullptr;     // stream(device index) -> handle of its current stream
  PyObject *workspace = nullptr;  // workspace(device index, stream, bytes) -> uint8 tensor
};
inline Bound lib;

#define BAD_IF(cond, ...) TORCH_CHECK_VALUE(!(cond), __VA_ARGS__)

// A Python callable was left with an exception.
struct PythonError {};

// A flag as Python reads it (its own exception where it has no truth value).
inline bool truth(PyObject *o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw PythonError{};
  return r == 1;
}

inline void *current_stream(const at::Device &dev) {
  PyObject *index = PyLong_FromLong(dev.index());
  PyObject *r = index ? PyObject_CallOneArg(lib.stream, index) : nullptr;
  Py_XDECREF(index);
  if (!r) throw PythonError{};
  void *s = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  if (!s && PyErr_Occurred()) throw PythonError{};
  return s;
}

// A call's kernels go into its stream together: threads that share a stream
// share its workspace, which the second kernel of a scan must find as the first
// one left it.
inline std::mutex enqueue;

// An error code becomes the binding's exception.
inline void check(int rc) {
  if (rc == GDN_OK) return;
  PyObject *r = PyObject_CallFunction(lib.raise, "i", rc);
  Py_XDECREF(r);
  if (r) PyErr_SetString(PyExc_RuntimeError, "the library returned an error code");
  throw PythonError{};
}

// Launches with the tensors' device current.
template <typename F> void launch(const at::Device &dev, F f) {
  const c10::DeviceGuard guard(dev);
  void *stream = current_stream(dev);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  {
    const std::lock_guard<std::mutex> lock(enqueue);
    rc = f(stream);
  }
  Py_END_ALLOW_THREADS;
  check(rc);
}

// --------------------------------------------------------------------- tensors

inline const Tensor &tensor(const char *name, PyObject *o) {
  BAD_IF(!THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
// An optional tensor on `dev`: NULL for None.
inline const Tensor *optional(const char *name, PyObject *o, const at::Device &dev) {
  if (o == Py_None) return nullptr;
  const Tensor &t = tensor(name, o);
  BAD_IF(t.device() != dev, name, " must be on ", dev);
  return &t;
}

inline void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

inline int float_type(at::ScalarType t) {
  return t == at::kFloat ? GDN_F32 : t == at::kBFloat16 ? GDN_BF16 : t == at::kHalf ? GDN_F16 : -1;
}
inline int state_type(at::ScalarType t) {
  if (t == at::kFloat8_e4m3fn) return GDN_FP8_E4M3;
  return t == at::kFloat8_e5m2 ? GDN_FP8_E5M2 : float_type(t);
}
inline int index_type(const char *name, const Tensor &t) {
  BAD_IF(t.scalar_type() != at::kInt && t.scalar_type() != at::kLong, name,
         " must be int32 or int64");
  BAD_IF(t.dim() != 1 || !t.is_contiguous(), name, " must be a contiguous 1-D tensor");
  BAD_IF(t.numel() > INT32_MAX, name, " is too long");
  return t.scalar_type() == at::kLong ? GDN_I64 : GDN_I32;
}

// Refuses a tensor whose derivatives the call would drop without a word: one that
// requires a gradient while gradients are recorded, or a dual tensor of forward
// mode.
inline void no_derivative(const char *name, const Tensor &t) {
  if (!t.unsafeGetTensorImpl()->autograd_meta()) return;  // neither, as for most tensors
  BAD_IF(c10::GradMode::is_enabled() && t.requires_grad(), name,
         " requires a gradient, but this call is not differentiable; use torch.no_grad()");
  BAD_IF(c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined(), name,
         " has a tangent, but there is no forward-mode derivative");
}

// The tensors that a call writes, for autograd: as with torch's own in-place
// operators on leaves, one that requires a gradient is refused, and after the
// launch their versions advance, so that a graph that saved one of them raises instead of
// using what is there now.
struct Writes {
  c10::SmallVector<const Tensor *, 8> all;

  void add(const char *name, const Tensor &t) {
    no_derivative(name, t);
    all.push_back(&t);
  }
  void add(const char *name, const Tensor *t) {
    if (t) add(name, *t);
  }
  void done() const {
    for (const Tensor *t : all) advance(*t);
  }
  static void advance(const Tensor &t) {  // (an inference tensor has no version)
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
};

inline void *status_word(PyObject *o, const at::Device &dev, Writes &writes) {
  const Tensor *t = optional("status", o, dev);
  BAD_IF(t && (t->scalar_type() != at::kInt || t->numel() < 1), "status must be an int32 tensor");
  writes.add("status", t);
  return ptr(t);
}

// A dimension of extent > 1 with stride 0: its elements alias.
inline bool expanded(const Tensor &t) {
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) > 1 && t.stride(i) == 0) return true;
  return false;
}

// Distance in elements of the first dimension's entries, each of which holds
// `inner` contiguous values.
inline int64_t row_stride(const char *name, const Tensor &t, int64_t inner) {
  if (t.numel() == 0) return inner;  // (contiguous() keeps an empty tensor's strides)
  int64_t want = 1;
  for (int64_t i = t.dim() - 1; i > 0; --i) {
    BAD_IF(t.size(i) > 1 && t.stride(i) != want, name,
           ": the values of one entry must be contiguous");
    want *= t.size(i);
  }
  if (t.size(0) <= 1) return inner;
  BAD_IF(t.stride(0) < inner, name, " must not overlap itself (stride ", t.stride(0), " < ", inner,
         ")");
  return t.stride(0);
}

inline void exactly(const char *name, const Tensor &t, at::IntArrayRef shape, at::ScalarType type) {
  BAD_IF(t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous(), name,
         " must be contiguous ", shape, " ", type);
}

inline Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Device &dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

inline PyObject *give(const Tensor &t) { return THPVariable_Wrap(t); }
inline PyObject *give_or_none(bool have, const Tensor &t) {
  if (have) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
inline PyObject *pack(std::initializer_list<PyObject *> items) {
  PyObject *r = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject *o : items) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

// The caller's workspace if it is large enough, else the binding's own for the
// current stream (kept in `memory`).
inline void *workspace_for(PyObject *o, size_t need, const at::Device &dev, Tensor &memory,
                           size_t &bytes) {
  if (o != Py_None) {
    const Tensor &t = tensor("workspace", o);
    BAD_IF(t.device() != dev || t.scalar_type() != at::kByte || !t.is_contiguous(),
           "workspace must be a contiguous uint8 tensor on ", dev);
    if ((size_t)t.numel() >= need) {
      bytes = (size_t)t.numel();
      return t.data_ptr();
    }
  }
  bytes = 0;
  if (need == 0) return nullptr;
  const c10::DeviceGuard guard(dev);
  PyObject *r = PyObject_CallFunction(lib.workspace, "iKn", (int)dev.index(),
                                      (unsigned long long)(uintptr_t)current_stream(dev),
                                      (Py_ssize_t)need);
  if (!r) throw PythonError{};
  const bool ok = THPVariable_Check(r);
  if (ok) memory = THPVariable_Unpack(r);
  Py_DECREF(r);
  BAD_IF(!ok, "no workspace");
  bytes = (size_t)memory.numel();
  return memory.data_ptr();
}

struct PoolView {
  int dtype;
  int64_t rows, strides[4], extent[3];
  void *data;

  PoolView(const char *name, const Tensor &t, bool written) {
    BAD_IF(!t.is_cuda(), name, " must be a device tensor");
    BAD_IF(t.dim() < 2 || t.dim() > 4, name,
           " must be [rows, ...] with one to three state dimensions");
    dtype = state_type(t.scalar_type());
    BAD_IF(dtype < 0, "unsupported ", name, " dtype");
    BAD_IF(written && expanded(t), name, " must not be an expanded view (a stride of 0 on a "
                                         "dimension of extent > 1)");
    rows = t.size(0);
    // a dimension of extent 1 is never stepped over; 1 keeps all-zero strides
    // (contiguous in the C ABI) out
    const int pad = 4 - (int)t.dim();
    for (int i = 0; i < 4; ++i) strides[i] = 1;
    for (int i = 0; i < 3; ++i) extent[i] = 1;
    if (rows > 1) strides[0] = t.stride(0);
    for (int64_t i = 1; i < t.dim(); ++i) {
      extent[pad + i - 1] = t.size(i);
      BAD_IF(t.size(i) == 0, name, " has empty rows");
      if (t.size(i) > 1) strides[pad + i] = t.stride(i);
    }
    data = t.data_ptr();
  }
};

inline const Tensor &row_list(const char *name, PyObject *o, const at::Device &dev) {
  const Tensor &t = tensor(name, o);
  BAD_IF(t.device() != dev, name, " must be a tensor on ", dev);
  return t;
}

// The layers' operators (torch_layer_calls.cpp); arguments as listed there.
PyObject *conv_forward(PyObject *const *a);
PyObject *conv_backward(PyObject *const *a);
PyObject *conv_decode(PyObject *const *a);
PyObject *scan_forward(PyObject *const *a);
PyObject *scan_backward(PyObject *const *a);
PyObject *scan_decode(PyObject *const *a);
PyObject *beam_select(PyObject *const *a);
PyObject *pool_reorder(PyObject *const *a);

}  // namespace calls
