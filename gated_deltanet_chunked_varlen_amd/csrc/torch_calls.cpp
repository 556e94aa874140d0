// torch_calls.cpp -- tensors to parameter blocks for the operators whose
// kernels run for a few microseconds (the gated linear recurrence and the
// state-pool rows), as a CPython module.
//
// From Python the same marshalling takes 4 to 15 us a call (an attribute of a
// tensor costs 70 to 150 ns there), more than the kernels it launches; here it
// takes a fraction of one.  Argument checks and memory only: every step of the
// computation is behind the C ABI, whose entry points this module gets as
// addresses (bind), so that it works with whichever build of the library is
// loaded.  What is wrong with an argument raises ValueError.
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

namespace {

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
  PyObject *raise = nullptr;      // raise(code): the exception of an error code
  PyObject *stream = nullptr;     // stream(device index) -> handle of its current stream
  PyObject *workspace = nullptr;  // workspace(device index, stream, bytes) -> uint8 tensor
} lib;

#define BAD_IF(cond, ...) TORCH_CHECK_VALUE(!(cond), __VA_ARGS__)

// A Python callable was left with an exception.
struct PythonError {};

// A flag as Python reads it (its own exception where it has no truth value).
bool truth(PyObject *o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw PythonError{};
  return r == 1;
}

void *current_stream(const at::Device &dev) {
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
std::mutex enqueue;

// An error code becomes the binding's exception.
void check(int rc) {
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

const Tensor &tensor(const char *name, PyObject *o) {
  BAD_IF(!THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
// An optional tensor on `dev`: NULL for None.
const Tensor *optional(const char *name, PyObject *o, const at::Device &dev) {
  if (o == Py_None) return nullptr;
  const Tensor &t = tensor(name, o);
  BAD_IF(t.device() != dev, name, " must be on ", dev);
  return &t;
}

void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

int float_type(at::ScalarType t) {
  return t == at::kFloat ? GDN_F32 : t == at::kBFloat16 ? GDN_BF16 : t == at::kHalf ? GDN_F16 : -1;
}
int state_type(at::ScalarType t) {
  if (t == at::kFloat8_e4m3fn) return GDN_FP8_E4M3;
  return t == at::kFloat8_e5m2 ? GDN_FP8_E5M2 : float_type(t);
}
int index_type(const char *name, const Tensor &t) {
  BAD_IF(t.scalar_type() != at::kInt && t.scalar_type() != at::kLong, name,
         " must be int32 or int64");
  BAD_IF(t.dim() != 1 || !t.is_contiguous(), name, " must be a contiguous 1-D tensor");
  BAD_IF(t.numel() > INT32_MAX, name, " is too long");
  return t.scalar_type() == at::kLong ? GDN_I64 : GDN_I32;
}

// Refuses a tensor whose derivatives the call would drop without a word: one that
// requires a gradient while gradients are recorded, or a dual tensor of forward
// mode.
void no_derivative(const char *name, const Tensor &t) {
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

void *status_word(PyObject *o, const at::Device &dev, Writes &writes) {
  const Tensor *t = optional("status", o, dev);
  BAD_IF(t && (t->scalar_type() != at::kInt || t->numel() < 1), "status must be an int32 tensor");
  writes.add("status", t);
  return ptr(t);
}

// A dimension of extent > 1 with stride 0: its elements alias.
bool expanded(const Tensor &t) {
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) > 1 && t.stride(i) == 0) return true;
  return false;
}

// Distance in elements of the first dimension's entries, each of which holds
// `inner` contiguous values.
int64_t row_stride(const char *name, const Tensor &t, int64_t inner) {
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

void exactly(const char *name, const Tensor &t, at::IntArrayRef shape, at::ScalarType type) {
  BAD_IF(t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous(), name,
         " must be contiguous ", shape, " ", type);
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Device &dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

PyObject *give(const Tensor &t) { return THPVariable_Wrap(t); }
PyObject *give_or_none(bool have, const Tensor &t) {
  if (have) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
PyObject *pack(std::initializer_list<PyObject *> items) {
  PyObject *r = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject *o : items) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

// ------------------------------------------------------------------ recurrence

struct Rec {
  gdn_recurrence_params p{};
  const Tensor &x, &g;
  at::Device dev;
  int64_t T, H, D, N = 1;
  Writes writes;
  Tensor init_copy;  // an expanded initial state, made contiguous
  Tensor memory;

  Rec(PyObject *x_, PyObject *g_, PyObject *cu_, bool decode)
      : x(tensor("x", x_)), g(tensor("g", g_)), dev(x.device()) {
    BAD_IF(!x.is_cuda(), "x must be a device tensor");
    no_derivative("x", x);
    no_derivative("g", g);
    BAD_IF(g.device() != dev, "g must be on ", dev);
    BAD_IF(x.dim() != 3, "x must be [total_seq_len, heads, head_size]");
    p.x_dtype = float_type(x.scalar_type());
    BAD_IF(p.x_dtype < 0, "x must be float32, bfloat16 or float16");
    BAD_IF(g.scalar_type() != at::kFloat && g.scalar_type() != x.scalar_type(),
           "g must be float32 or x's dtype");
    p.g_dtype = float_type(g.scalar_type());
    T = x.size(0);
    H = x.size(1);
    D = x.size(2);
    const bool per_head = g.dim() == 2;
    BAD_IF(!(per_head || (g.dim() == 3 && g.size(2) == D)) || g.size(0) != T || g.size(1) != H,
           "g must be [", T, ", ", H, ", ", D, "] or [", T, ", ", H, "]");
    BAD_IF(H < 1 || D < 1, "x needs at least one head and one channel");
    BAD_IF(H > INT32_MAX || D > INT32_MAX || T > INT32_MAX, "x is too large");
    p.total_tokens = T;
    p.num_heads = (int32_t)H;
    p.head_size = (int32_t)D;
    p.g_per_head = per_head;
    p.x = x.data_ptr();
    p.g = g.data_ptr();
    p.x_stride = row_stride("x", x, H * D);
    p.g_stride = row_stride("g", g, per_head ? H : H * D);
    if (decode) {
      N = T;
    } else if (const Tensor *cu = optional("cu_seqlens", cu_, dev)) {
      p.cu_seqlens_type = index_type("cu_seqlens", *cu);
      BAD_IF(cu->numel() < 1, "cu_seqlens must hold at least one offset");
      p.cu_seqlens = cu->data_ptr();
      N = cu->numel() - 1;
    }
    p.num_seqs = (int32_t)N;
  }

  Tensor like_x() const { return fresh({T, H, D}, x.scalar_type(), dev); }
  Tensor states(int64_t rows) const { return fresh({rows, H, D}, at::kFloat, dev); }

  void check_state(const char *name, const Tensor &t, int64_t rows) const {
    BAD_IF(state_type(t.scalar_type()) < 0, "unsupported ", name, " dtype");
    BAD_IF(t.dim() != 3 || t.size(0) != rows || t.size(1) != H || t.size(2) != D, name,
           " must be [", rows, ", ", H, ", ", D, "]");
  }

  void initial(const Tensor *t, int64_t rows) {
    if (!t) return;
    check_state("initial_state", *t, rows);
    no_derivative("initial_state", *t);
    if (expanded(*t)) {
      init_copy = t->contiguous();
      t = &init_copy;
    }
    p.initial_state = t->data_ptr();
    p.initial_state_dtype = state_type(t->scalar_type());
    p.initial_state_stride = row_stride("initial_state", *t, H * D);
  }

  // Initial, final and pool states of a forward or decode call; returns the
  // final state's tensor (undefined without one).
  Tensor forward_states(PyObject *init_, bool with_final, PyObject *out_, PyObject *idx_) {
    const Tensor *init = optional("initial_state", init_, dev);
    const Tensor *out = optional("output_state", out_, dev);
    const Tensor *idx = optional("state_indices", idx_, dev);
    int64_t rows = N;
    if (idx) {
      p.state_indices_type = index_type("state_indices", *idx);
      BAD_IF(idx->numel() != N, "state_indices must hold ", N, " rows");
      const Tensor *pool = out ? out : init;
      BAD_IF(!pool, "state_indices needs a state pool");
      BAD_IF(pool->dim() < 1, "a state pool must be [rows, heads, head_size]");
      p.state_indices = idx->data_ptr();
      p.pool_size = rows = pool->size(0);
    }
    initial(init, rows);
    if (!with_final) return Tensor();
    BAD_IF(!out && idx, "output_state (the pool) is required with state_indices");
    writes.add("output_state", out);
    Tensor fin = out ? *out : states(N);
    check_state("output_state", fin, rows);
    BAD_IF(expanded(fin), "output_state must not be an expanded view (a stride of 0 on a "
                          "dimension of extent > 1)");
    p.output_final_state = 1;
    p.output_state = fin.data_ptr();
    p.output_state_dtype = state_type(fin.scalar_type());
    p.output_state_stride = row_stride("output_state", fin, H * D);
    return fin;
  }

  Tensor output(PyObject *o) {
    const Tensor *t = optional("output", o, dev);
    if (t) exactly("output", *t, x.sizes(), x.scalar_type());
    writes.add("output", t);
    Tensor out = t ? *t : like_x();
    p.output = out.data_ptr();
    return out;
  }

  std::vector<int64_t> chunk_shape() const {
    return {(T + GDN_RECURRENCE_CHUNK - 1) / GDN_RECURRENCE_CHUNK, H, D};
  }

  // The caller's workspace if it is large enough, else the binding's own for
  // the current stream.
  void take_workspace(PyObject *o, bool backward) {
    const size_t need = lib.rec_workspace(&p, backward);
    if (o != Py_None) {
      const Tensor &t = tensor("workspace", o);
      BAD_IF(t.device() != dev || t.scalar_type() != at::kByte || !t.is_contiguous(),
             "workspace must be a contiguous uint8 tensor on ", dev);
      if ((size_t)t.numel() >= need) {
        p.workspace = t.data_ptr();
        p.workspace_bytes = (size_t)t.numel();
        return;
      }
    }
    if (need == 0) return;
    const c10::DeviceGuard guard(dev);
    PyObject *r = PyObject_CallFunction(lib.workspace, "iKn", (int)dev.index(),
                                        (unsigned long long)(uintptr_t)current_stream(dev),
                                        (Py_ssize_t)need);
    if (!r) throw PythonError{};
    const bool ok = THPVariable_Check(r);
    if (ok) memory = THPVariable_Unpack(r);
    Py_DECREF(r);
    BAD_IF(!ok, "no workspace");
    p.workspace = memory.data_ptr();
    p.workspace_bytes = (size_t)memory.numel();
  }
};

// (x, g, initial_state, output_final_state, cu_seqlens, output, output_state,
//  state_indices, return_chunk_states, status, workspace)
// -> (output, final state or None, chunk states or None)
PyObject *rec_forward(PyObject *const *a) {
  Rec r(a[0], a[1], a[4], false);
  const bool with_final = truth(a[3]), keep = truth(a[8]);
  const Tensor out = r.output(a[5]);
  const Tensor fin = r.forward_states(a[2], with_final, a[6], a[7]);
  r.p.status = (int32_t *)status_word(a[9], r.dev, r.writes);
  Tensor kept;
  if (keep) {
    kept = fresh(r.chunk_shape(), at::kFloat, r.dev);
    r.p.chunk_states = (float *)kept.data_ptr();
  }
  r.take_workspace(a[10], false);
  launch(r.dev, [&](void *s) { return lib.rec_forward(&r.p, s); });
  r.writes.done();
  return pack({give(out), give_or_none(with_final, fin), give_or_none(keep, kept)});
}

// (doutput, x, g, initial_state, dfinal_state, cu_seqlens, chunk_states,
//  output_dinitial_state, dx, dg, dinitial_state, status, workspace)
// -> (dx, dg) or (dx, dg, dinitial_state)
PyObject *rec_backward(PyObject *const *a) {
  Rec r(a[1], a[2], a[5], false);
  const Tensor &dout = tensor("doutput", a[0]);
  BAD_IF(dout.device() != r.dev, "doutput must be on ", r.dev);
  BAD_IF(dout.scalar_type() != r.x.scalar_type() || dout.sizes() != r.x.sizes(),
         "doutput must have x's shape and dtype");
  no_derivative("doutput", dout);
  r.p.doutput = dout.data_ptr();
  r.p.doutput_stride = row_stride("doutput", dout, r.H * r.D);
  r.initial(optional("initial_state", a[3], r.dev), r.N);
  const std::vector<int64_t> rows = {r.N, r.H, r.D};
  auto buffer = [&](const char *name, PyObject *o, at::IntArrayRef shape, at::ScalarType type) {
    const Tensor *t = optional(name, o, r.dev);
    if (t) exactly(name, *t, shape, type);
    if (t) no_derivative(name, *t);
    return t;
  };
  r.p.dfinal_state = (const float *)ptr(buffer("dfinal_state", a[4], rows, at::kFloat));
  r.p.chunk_states = (float *)ptr(buffer("chunk_states", a[6], r.chunk_shape(), at::kFloat));
  const bool with_init = truth(a[7]);
  const Tensor *dx_ = buffer("dx", a[8], r.x.sizes(), r.x.scalar_type());
  const Tensor *dg_ = buffer("dg", a[9], r.g.sizes(), r.g.scalar_type());
  const Tensor *di_ = buffer("dinitial_state", a[10], rows, at::kFloat);
  r.writes.add("dx", dx_);
  r.writes.add("dg", dg_);
  if (with_init) r.writes.add("dinitial_state", di_);
  r.p.status = (int32_t *)status_word(a[11], r.dev, r.writes);
  const Tensor dx = dx_ ? *dx_ : r.like_x();
  const Tensor dg = dg_ ? *dg_ : fresh(r.g.sizes(), r.g.scalar_type(), r.dev);
  r.p.dx = dx.data_ptr();
  r.p.dg = dg.data_ptr();
  Tensor di;
  if (with_init) {
    di = di_ ? *di_ : r.states(r.N);
    r.p.dinitial_state = (float *)di.data_ptr();
  }
  r.take_workspace(a[12], true);
  launch(r.dev, [&](void *s) { return lib.rec_backward(&r.p, s); });
  r.writes.done();
  return with_init ? pack({give(dx), give(dg), give(di)}) : pack({give(dx), give(dg)});
}

// (x, g, initial_state, output_final_state, output, output_state,
//  state_indices, status) -> output or (output, final state)
PyObject *rec_decode(PyObject *const *a) {
  Rec r(a[0], a[1], Py_None, true);
  const bool with_final = truth(a[3]);
  const Tensor out = r.output(a[4]);
  const Tensor fin = r.forward_states(a[2], with_final, a[5], a[6]);
  r.p.status = (int32_t *)status_word(a[7], r.dev, r.writes);
  launch(r.dev, [&](void *s) { return lib.rec_decode(&r.p, s); });
  r.writes.done();
  return with_final ? pack({give(out), give(fin)}) : give(out);
}

// ----------------------------------------------------------------------- pools

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

void set_destination(gdn_pool_params &p, const PoolView &v) {
  for (int i = 0; i < 3; ++i) p.extent[i] = v.extent[i];
  for (int i = 0; i < 4; ++i) p.dst_strides[i] = v.strides[i];
  p.dst = v.data;
  p.dst_dtype = v.dtype;
  p.dst_pool_rows = v.rows;
}

const Tensor &row_list(const char *name, PyObject *o, const at::Device &dev) {
  const Tensor &t = tensor(name, o);
  BAD_IF(t.device() != dev, name, " must be a tensor on ", dev);
  return t;
}

// (pool, src_rows, dst_rows, src_pool, status) -> pool
PyObject *pool_copy(PyObject *const *a) {
  const Tensor &pool = tensor("pool", a[0]);
  const at::Device dev = pool.device();
  const Tensor &src_rows = row_list("src_rows", a[1], dev);
  const Tensor &dst_rows = row_list("dst_rows", a[2], dev);
  gdn_pool_params p{};
  const PoolView to("pool", pool, true);
  set_destination(p, to);
  p.rows_type = index_type("src_rows", src_rows);
  BAD_IF(index_type("dst_rows", dst_rows) != p.rows_type,
         "src_rows and dst_rows must share a dtype");
  BAD_IF(src_rows.numel() != dst_rows.numel(),
         "src_rows and dst_rows must have the same length");
  Writes writes;
  writes.add("pool", pool);
  p.status = (int32_t *)status_word(a[4], dev, writes);
  Tensor from = a[3] == Py_None ? pool : tensor("src_pool", a[3]);
  BAD_IF(from.device() != dev, "src_pool must be on ", dev);
  no_derivative("src_pool", from);
  if (expanded(from)) from = from.contiguous();
  const PoolView v("src_pool", from, false);
  for (int i = 0; i < 3; ++i)
    BAD_IF(v.extent[i] != to.extent[i], "rows of pool and src_pool differ in shape");
  for (int i = 0; i < 4; ++i) p.src_strides[i] = v.strides[i];
  p.src = v.data;
  p.src_dtype = v.dtype;
  p.src_pool_rows = v.rows;
  p.src_rows = src_rows.data_ptr();
  p.dst_rows = dst_rows.data_ptr();
  p.count = dst_rows.numel();
  if (v.rows == 0 || to.rows == 0) {
    BAD_IF(p.count > 0, "a pool without rows cannot be copied from or into");
  } else {
    launch(dev, [&](void *s) { return lib.pool_copy(&p, s); });
    writes.done();
  }
  Py_INCREF(a[0]);
  return a[0];
}

// (pool, rows, status) -> pool
PyObject *pool_reset(PyObject *const *a) {
  const Tensor &pool = tensor("pool", a[0]);
  const Tensor &rows = row_list("rows", a[1], pool.device());
  gdn_pool_params p{};
  set_destination(p, PoolView("pool", pool, true));
  p.rows_type = index_type("rows", rows);
  Writes writes;
  writes.add("pool", pool);
  p.status = (int32_t *)status_word(a[2], pool.device(), writes);
  p.dst_rows = rows.data_ptr();
  p.count = rows.numel();
  launch(pool.device(), [&](void *s) { return lib.pool_reset(&p, s); });
  writes.done();
  Py_INCREF(a[0]);
  return a[0];
}

// (list of pools, state_indices, output_indices, row_map, status)
// -> (renamed indices, num_live)
PyObject *pool_compact(PyObject *const *a) {
  const Py_ssize_t n = PyList_Check(a[0]) ? PyList_GET_SIZE(a[0]) : 0;
  BAD_IF(n < 1, "state_pool_compact needs a pool");
  const Tensor &first = tensor("pool", PyList_GET_ITEM(a[0], 0));
  const at::Device dev = first.device();
  const Tensor &idx = row_list("state_indices", a[1], dev);
  const int kind = index_type("state_indices", idx);
  const Tensor *out_ = optional("output_indices", a[2], dev);
  BAD_IF(out_ && (out_->scalar_type() != idx.scalar_type() || out_->sizes() != idx.sizes() ||
                  !out_->is_contiguous()),
         "output_indices must match state_indices");
  const Tensor *map = optional("row_map", a[3], dev);
  BAD_IF(map && (map->scalar_type() != at::kInt || map->dim() != 1 || first.dim() < 1 ||
                 map->size(0) != first.size(0) || !map->is_contiguous()),
         "row_map must be contiguous int32 [rows] on ", dev);
  Writes writes;
  writes.add("output_indices", out_);
  writes.add("row_map", map);
  int32_t *status = (int32_t *)status_word(a[4], dev, writes);
  std::vector<gdn_pool_params> calls((size_t)n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const Tensor &pool = tensor("pool", PyList_GET_ITEM(a[0], i));
    BAD_IF(pool.device() != dev, "pools must share a device");
    writes.add("pool", pool);
    gdn_pool_params p{};
    set_destination(p, PoolView("pool", pool, true));
    BAD_IF(pool.size(0) != first.size(0), "pools must share a number of rows");
    p.rows_type = kind;
    p.status = status;
    p.dst_rows = idx.data_ptr();
    p.count = idx.numel();
    check(lib.pool_validate(&p, 2));  // every pool before the first is moved
    calls[(size_t)i] = p;
  }
  const Tensor out = out_ ? *out_ : fresh(idx.sizes(), idx.scalar_type(), dev);
  const Tensor live = fresh({1}, at::kInt, dev);
  for (const gdn_pool_params &p : calls)
    launch(dev, [&](void *s) {
      return lib.pool_compact(&p, out.data_ptr(), (int32_t *)live.data_ptr(), (int32_t *)ptr(map),
                              s);
    });
  writes.done();
  return pack({give(out), give(live)});
}

// ---------------------------------------------------------------------- module

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", N, n);
    return nullptr;
  }
  if (!lib.raise) {
    PyErr_SetString(PyExc_ImportError, "the library is not bound");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PythonError &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// advance_versions(tensors or None ...): what other calls have written.
PyObject *advance_versions(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  for (Py_ssize_t i = 0; i < n; ++i)
    if (a[i] != Py_None) Writes::advance(tensor("a written buffer", a[i]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// bind(eight addresses, raise, stream, workspace)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  constexpr int kEntries = 8;
  if (n != kEntries + 3) {
    PyErr_SetString(PyExc_TypeError, "eleven arguments expected");
    return nullptr;
  }
  void *f[kEntries];
  for (int i = 0; i < kEntries; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a NULL entry point");
      return nullptr;
    }
  }
  lib.rec_workspace = (decltype(lib.rec_workspace))f[0];
  lib.rec_forward = (decltype(lib.rec_forward))f[1];
  lib.rec_backward = (decltype(lib.rec_backward))f[2];
  lib.rec_decode = (decltype(lib.rec_decode))f[3];
  lib.pool_copy = (decltype(lib.pool_copy))f[4];
  lib.pool_reset = (decltype(lib.pool_reset))f[5];
  lib.pool_compact = (decltype(lib.pool_compact))f[6];
  lib.pool_validate = (decltype(lib.pool_validate))f[7];
  for (int i = kEntries; i < kEntries + 3; ++i) Py_INCREF(a[i]);
  lib.stream = a[kEntries + 1];
  lib.workspace = a[kEntries + 2];
  lib.raise = a[kEntries];
  Py_RETURN_NONE;
}

#define CALL(name, f, n) {name, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"advance_versions", (PyCFunction)(void (*)(void))advance_versions, METH_FASTCALL, nullptr},
    CALL("rec_forward", rec_forward, 11),
    CALL("rec_backward", rec_backward, 13),
    CALL("rec_decode", rec_decode, 8),
    CALL("pool_copy", pool_copy, 5),
    CALL("pool_reset", pool_reset, 3),
    CALL("pool_compact", pool_compact, 5),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module_def); }
