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
#include "torch_calls.h"

namespace {

using namespace calls;

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

  void take_workspace(PyObject *o, bool backward) {
    p.workspace = workspace_for(o, lib.rec_workspace(&p, backward), dev, memory, p.workspace_bytes);
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

void set_destination(gdn_pool_params &p, const PoolView &v) {
  for (int i = 0; i < 3; ++i) p.extent[i] = v.extent[i];
  for (int i = 0; i < 4; ++i) p.dst_strides[i] = v.strides[i];
  p.dst = v.data;
  p.dst_dtype = v.dtype;
  p.dst_pool_rows = v.rows;
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

// bind(addresses in the order below, raise, stream, workspace)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  constexpr int kEntries = 20;
  if (n != kEntries + 3) {
    PyErr_SetString(PyExc_TypeError, "twenty addresses and three callables expected");
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
  lib.conv_workspace = (decltype(lib.conv_workspace))f[8];
  lib.conv_forward = (decltype(lib.conv_forward))f[9];
  lib.conv_backward = (decltype(lib.conv_backward))f[10];
  lib.conv_decode = (decltype(lib.conv_decode))f[11];
  lib.scan_chunk = (decltype(lib.scan_chunk))f[12];
  lib.scan_workspace = (decltype(lib.scan_workspace))f[13];
  lib.scan_forward = (decltype(lib.scan_forward))f[14];
  lib.scan_backward = (decltype(lib.scan_backward))f[15];
  lib.scan_decode = (decltype(lib.scan_decode))f[16];
  lib.beam_workspace = (decltype(lib.beam_workspace))f[17];
  lib.beam_select = (decltype(lib.beam_select))f[18];
  lib.pool_reorder = (decltype(lib.pool_reorder))f[19];
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
    CALL("conv_forward", calls::conv_forward, 12),
    CALL("conv_backward", calls::conv_backward, 15),
    CALL("conv_decode", calls::conv_decode, 10),
    CALL("scan_forward", calls::scan_forward, 18),
    CALL("scan_backward", calls::scan_backward, 17),
    CALL("scan_decode", calls::scan_decode, 15),
    CALL("beam_select", calls::beam_select, 4),
    CALL("pool_reorder", calls::pool_reorder, 5),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module_def); }
