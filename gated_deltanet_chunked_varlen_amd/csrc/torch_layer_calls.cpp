// torch_layer_calls.cpp -- tensors to parameter blocks for the short convolution,
// the selective scan and beam search.
#include "torch_calls.h"

namespace calls {

namespace {

// The tensors of a call on a packed batch; P: its parameter block.
template <typename P> struct Packed {
  P p{};
  const Tensor &x;
  at::Device dev;
  int64_t T, C, N = 1;
  Writes writes;
  Tensor init_copy;  // an expanded initial state, made contiguous
  Tensor memory;
  std::vector<int64_t> row;  // shape of a state

  explicit Packed(PyObject *x_) : x(tensor("x", x_)), dev(x.device()) {
    BAD_IF(!x.is_cuda(), "x must be a device tensor");
    BAD_IF(x.dim() != 2, "x must be [total_seq_len, channels]");
    no_derivative("x", x);
    p.x_dtype = float_type(x.scalar_type());
    BAD_IF(p.x_dtype < 0, "x must be float32, bfloat16 or float16");
    T = x.size(0);
    C = x.size(1);
    BAD_IF(C < 1, "x needs at least one channel");
    BAD_IF(T > INT32_MAX || C > INT32_MAX, "x is too large");
    p.total_tokens = T;
    p.channels = (int32_t)C;
    p.x = x.data_ptr();
    p.x_stride = row_stride("x", x, C);
  }

  void batch(PyObject *cu_, bool decode) {
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

  int64_t row_size() const { return row[0] * row[1]; }
  std::vector<int64_t> rows(int64_t n) const { return {n, row[0], row[1]}; }

  // An input of x's shape and dtype, token rows contiguous.
  void *like_x(const char *name, const Tensor &t, int64_t &stride) const {
    BAD_IF(t.device() != dev, name, " must be on ", dev);
    BAD_IF(t.scalar_type() != x.scalar_type() || t.sizes() != x.sizes(), name,
           " must have x's shape and dtype");
    no_derivative(name, t);
    stride = row_stride(name, t, C);
    return t.data_ptr();
  }
  // An optional contiguous input.
  const Tensor *exact(const char *name, PyObject *o, at::IntArrayRef shape, at::ScalarType type) {
    const Tensor *t = optional(name, o, dev);
    if (t) exactly(name, *t, shape, type);
    if (t) no_derivative(name, *t);
    return t;
  }
  // An output: the caller's buffer or a new one.
  Tensor buffer(const char *name, PyObject *o, at::IntArrayRef shape, at::ScalarType type) {
    const Tensor *t = optional(name, o, dev);
    if (t) exactly(name, *t, shape, type);
    writes.add(name, t);
    return t ? *t : fresh(shape, type, dev);
  }

  void check_state(const char *name, const Tensor &t, int64_t n) const {
    BAD_IF(state_type(t.scalar_type()) < 0, "unsupported ", name, " dtype");
    BAD_IF(t.dim() != 3 || t.size(0) != n || t.size(1) != row[0] || t.size(2) != row[1], name,
           " must be [", n, ", ", row[0], ", ", row[1], "]");
  }

  void initial(const Tensor *t, int64_t n) {
    if (!t) return;
    check_state("initial_state", *t, n);
    no_derivative("initial_state", *t);
    if (expanded(*t)) {
      init_copy = t->contiguous();
      t = &init_copy;
    }
    p.initial_state = t->data_ptr();
    p.initial_state_dtype = state_type(t->scalar_type());
    p.initial_state_stride = row_stride("initial_state", *t, row_size());
  }

  // Initial, final and pool states of a forward or decode call; returns the
  // final state's tensor (undefined without one).
  Tensor states(PyObject *init_, bool with_final, PyObject *out_, PyObject *idx_) {
    const Tensor *init = optional("initial_state", init_, dev);
    const Tensor *out = optional("output_state", out_, dev);
    const Tensor *idx = optional("state_indices", idx_, dev);
    int64_t n = N;
    if (idx) {
      p.state_indices_type = index_type("state_indices", *idx);
      BAD_IF(idx->numel() != N, "state_indices must hold ", N, " rows");
      const Tensor *pool = out ? out : init;
      BAD_IF(!pool, "state_indices needs a state pool");
      BAD_IF(pool->dim() < 1, "a state pool must be [rows, ", row[0], ", ", row[1], "]");
      p.state_indices = idx->data_ptr();
      p.pool_size = n = pool->size(0);
    }
    initial(init, n);
    if (!with_final) return Tensor();
    BAD_IF(!out && idx, "output_state (the pool) is required with state_indices");
    writes.add("output_state", out);
    Tensor fin = out ? *out : fresh(rows(N), at::kFloat, dev);
    check_state("output_state", fin, n);
    BAD_IF(expanded(fin), "output_state must not be an expanded view (a stride of 0 on a "
                          "dimension of extent > 1)");
    p.output_final_state = 1;
    p.output_state = fin.data_ptr();
    p.output_state_dtype = state_type(fin.scalar_type());
    p.output_state_stride = row_stride("output_state", fin, row_size());
    return fin;
  }

  void status(PyObject *o) { p.status = (int32_t *)status_word(o, dev, writes); }
  void take_workspace(PyObject *o, size_t need) {
    p.workspace = workspace_for(o, need, dev, memory, p.workspace_bytes);
  }
  template <typename F> void run(F f) {
    launch(dev, [&](void *s) { return f(&p, s); });
    writes.done();
  }
};

// ---------------------------------------------------------------- convolution

struct Conv : Packed<gdn_convolution_params> {
  const Tensor &weight;
  const Tensor *bias;

  Conv(PyObject *x_, PyObject *w_, PyObject *bias_, PyObject *silu, PyObject *cu, bool decode)
      : Packed(x_), weight(tensor("weight", w_)), bias(optional("bias", bias_, dev)) {
    BAD_IF(weight.device() != dev, "weight must be on ", dev);
    BAD_IF(weight.scalar_type() != at::kFloat && weight.scalar_type() != x.scalar_type(),
           "weight must be float32 or x's dtype");
    BAD_IF(weight.dim() != 2 || weight.size(0) != C || weight.size(1) < 2 || weight.size(1) > 4 ||
               !weight.is_contiguous(),
           "weight must be contiguous [", C, ", width], width 2, 3 or 4");
    no_derivative("weight", weight);
    if (bias) {
      exactly("bias", *bias, {C}, weight.scalar_type());
      no_derivative("bias", *bias);
    }
    p.width = (int32_t)weight.size(1);
    p.weight_dtype = float_type(weight.scalar_type());
    p.weight = weight.data_ptr();
    p.bias = ptr(bias);
    p.silu = truth(silu);
    row = {weight.size(1) - 1, C};
    batch(cu, decode);
  }
};

// ----------------------------------------------------------------------- scan

struct Scan : Packed<gdn_scan_params> {
  const Tensor &B, &Cm;
  const Tensor *D, *dbias, *z;

  // a: x, delta, A, B, C, D, z, delta_bias, delta_softplus
  Scan(PyObject *const *a, PyObject *cu, bool decode)
      : Packed(a[0]), B(tensor("B", a[3])), Cm(tensor("C", a[4])), D(nullptr), dbias(nullptr),
        z(optional("z", a[6], dev)) {
    p.delta = like_x("delta", tensor("delta", a[1]), p.delta_stride);
    if (z) p.z = like_x("z", *z, p.z_stride);
    const Tensor &A = tensor("A", a[2]);
    BAD_IF(A.device() != dev, "A must be on ", dev);
    BAD_IF(A.dim() != 2 || A.size(0) != C || A.size(1) < 1 || A.size(1) > 64,
           "A must be [", C, ", states], 1 to 64 states");
    exactly("A", A, A.sizes(), at::kFloat);
    no_derivative("A", A);
    p.A = (const float *)A.data_ptr();
    p.num_states = (int32_t)A.size(1);
    row = {C, A.size(1)};
    BAD_IF(B.dim() != 3 || B.size(0) != T || B.size(1) < 1 || B.size(2) != A.size(1) ||
               C % B.size(1) != 0,
           "B must be [", T, ", groups, ", A.size(1), "], the groups a divisor of ", C);
    BAD_IF(Cm.sizes() != B.sizes(), "C must have B's shape");
    for (const Tensor *t : {&B, &Cm}) {
      BAD_IF(t->device() != dev || t->scalar_type() != x.scalar_type(),
             "B and C must have x's dtype and device");
      no_derivative("B or C", *t);
    }
    p.groups = (int32_t)B.size(1);
    p.b_stride = row_stride("B", B, B.size(1) * B.size(2));
    p.c_stride = row_stride("C", Cm, B.size(1) * B.size(2));
    p.B = B.data_ptr();
    p.C = Cm.data_ptr();
    D = exact("D", a[5], {C}, at::kFloat);
    dbias = exact("delta_bias", a[7], {C}, at::kFloat);
    p.D = (const float *)ptr(D);
    p.delta_bias = (const float *)ptr(dbias);
    p.delta_softplus = truth(a[8]);
    batch(cu, decode);
  }

  std::vector<int64_t> chunk_shape() const {
    const int64_t chunk = lib.scan_chunk(&p);
    BAD_IF(chunk < 1, "the call is too large");
    return {(T + chunk - 1) / chunk, row[1], C};
  }
};

}  // namespace

// (x, weight, bias, silu, initial_state, output_final_state, cu_seqlens, output,
//  output_state, state_indices, status, workspace) -> (output, final state or None)
PyObject *conv_forward(PyObject *const *a) {
  Conv r(a[0], a[1], a[2], a[3], a[6], false);
  const bool with_final = truth(a[5]);
  const Tensor out = r.buffer("output", a[7], r.x.sizes(), r.x.scalar_type());
  r.p.output = out.data_ptr();
  const Tensor fin = r.states(a[4], with_final, a[8], a[9]);
  r.status(a[10]);
  r.take_workspace(a[11], lib.conv_workspace(&r.p, 0));
  r.run(lib.conv_forward);
  return pack({give(out), give_or_none(with_final, fin)});
}

// (doutput, x, weight, bias, silu, initial_state, dfinal_state, cu_seqlens,
//  output_dinitial_state, dx, dweight, dbias, dinitial_state, status, workspace)
// -> (dx, dweight, dbias or None) or with dinitial_state behind them
PyObject *conv_backward(PyObject *const *a) {
  Conv r(a[1], a[2], a[3], a[4], a[7], false);
  r.p.doutput = r.like_x("doutput", tensor("doutput", a[0]), r.p.doutput_stride);
  r.initial(optional("initial_state", a[5], r.dev), r.N);
  r.p.dfinal_state = (const float *)ptr(r.exact("dfinal_state", a[6], r.rows(r.N), at::kFloat));
  const bool with_init = truth(a[8]);
  const Tensor dx = r.buffer("dx", a[9], r.x.sizes(), r.x.scalar_type());
  const Tensor dw = r.buffer("dweight", a[10], r.weight.sizes(), at::kFloat);
  Tensor db, di;
  BAD_IF(!r.bias && a[11] != Py_None, "dbias needs a bias");
  if (r.bias) db = r.buffer("dbias", a[11], r.bias->sizes(), at::kFloat);
  if (with_init) di = r.buffer("dinitial_state", a[12], r.rows(r.N), at::kFloat);
  r.p.dx = dx.data_ptr();
  r.p.dweight = (float *)dw.data_ptr();
  if (r.bias) r.p.dbias = (float *)db.data_ptr();
  if (with_init) r.p.dinitial_state = (float *)di.data_ptr();
  r.status(a[13]);
  r.take_workspace(a[14], lib.conv_workspace(&r.p, 1));
  r.run(lib.conv_backward);
  PyObject *bias = give_or_none(r.bias != nullptr, db);
  return with_init ? pack({give(dx), give(dw), bias, give(di)}) : pack({give(dx), give(dw), bias});
}

// (x, weight, bias, silu, initial_state, output_final_state, output,
//  output_state, state_indices, status) -> output or (output, final state)
PyObject *conv_decode(PyObject *const *a) {
  Conv r(a[0], a[1], a[2], a[3], Py_None, true);
  const bool with_final = truth(a[5]);
  const Tensor out = r.buffer("output", a[6], r.x.sizes(), r.x.scalar_type());
  r.p.output = out.data_ptr();
  const Tensor fin = r.states(a[4], with_final, a[7], a[8]);
  r.status(a[9]);
  r.run(lib.conv_decode);
  return with_final ? pack({give(out), give(fin)}) : give(out);
}

// (x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state,
//  output_final_state, cu_seqlens, output, output_state, state_indices,
//  return_chunk_states, status, workspace)
// -> (output, final state or None, chunk states or None)
PyObject *scan_forward(PyObject *const *a) {
  Scan r(a, a[11], false);
  const bool with_final = truth(a[10]), keep = truth(a[15]);
  const Tensor out = r.buffer("output", a[12], r.x.sizes(), r.x.scalar_type());
  r.p.output = out.data_ptr();
  const Tensor fin = r.states(a[9], with_final, a[13], a[14]);
  r.status(a[16]);
  Tensor kept;
  if (keep) {
    kept = fresh(r.chunk_shape(), at::kFloat, r.dev);
    r.p.chunk_states = (float *)kept.data_ptr();
  }
  r.take_workspace(a[17], lib.scan_workspace(&r.p, 0));
  r.run(lib.scan_forward);
  return pack({give(out), give_or_none(with_final, fin), give_or_none(keep, kept)});
}

// (doutput, x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state,
//  dfinal_state, cu_seqlens, chunk_states, output_dinitial_state, status,
//  workspace)
// -> (dx, ddelta, dA, dB, dC, dD, dz, ddelta_bias), None for what has no input,
//    or with dinitial_state behind them
PyObject *scan_backward(PyObject *const *a) {
  Scan r(a + 1, a[12], false);
  const at::ScalarType type = r.x.scalar_type();
  r.p.doutput = r.like_x("doutput", tensor("doutput", a[0]), r.p.doutput_stride);
  const Tensor *init = optional("initial_state", a[10], r.dev);
  BAD_IF(init && init->scalar_type() != at::kFloat, "initial_state must be float32");
  r.initial(init, r.N);
  r.p.dfinal_state = (const float *)ptr(r.exact("dfinal_state", a[11], r.rows(r.N), at::kFloat));
  if (a[13] != Py_None)
    r.p.chunk_states =
        (float *)ptr(r.exact("chunk_states", a[13], r.chunk_shape(), at::kFloat));
  const bool with_init = truth(a[14]);
  r.status(a[15]);
  const at::IntArrayRef shape = r.x.sizes();
  const Tensor dx = fresh(shape, type, r.dev), dd = fresh(shape, type, r.dev);
  const Tensor dA = fresh(r.row, at::kFloat, r.dev);
  const Tensor dB = fresh(r.B.sizes(), type, r.dev), dC = fresh(r.B.sizes(), type, r.dev);
  Tensor dD, dz, db, di;
  r.p.dx = dx.data_ptr();
  r.p.ddelta = dd.data_ptr();
  r.p.dA = (float *)dA.data_ptr();
  r.p.dB = dB.data_ptr();
  r.p.dC = dC.data_ptr();
  if (r.D) r.p.dD = (float *)(dD = fresh({r.C}, at::kFloat, r.dev)).data_ptr();
  if (r.z) r.p.dz = (dz = fresh(shape, type, r.dev)).data_ptr();
  if (r.dbias) r.p.ddelta_bias = (float *)(db = fresh({r.C}, at::kFloat, r.dev)).data_ptr();
  if (with_init)
    r.p.dinitial_state = (float *)(di = fresh(r.rows(r.N), at::kFloat, r.dev)).data_ptr();
  r.take_workspace(a[16], lib.scan_workspace(&r.p, 1));
  r.run(lib.scan_backward);
  PyObject *oD = give_or_none(r.D != nullptr, dD), *oz = give_or_none(r.z != nullptr, dz);
  PyObject *ob = give_or_none(r.dbias != nullptr, db);
  if (with_init)
    return pack({give(dx), give(dd), give(dA), give(dB), give(dC), oD, oz, ob, give(di)});
  return pack({give(dx), give(dd), give(dA), give(dB), give(dC), oD, oz, ob});
}

// (x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state,
//  output_final_state, output, output_state, state_indices, status)
// -> output or (output, final state)
PyObject *scan_decode(PyObject *const *a) {
  Scan r(a, Py_None, true);
  const bool with_final = truth(a[10]);
  const Tensor out = r.buffer("output", a[11], r.x.sizes(), r.x.scalar_type());
  r.p.output = out.data_ptr();
  const Tensor fin = r.states(a[9], with_final, a[12], a[13]);
  r.status(a[14]);
  r.run(lib.scan_decode);
  return with_final ? pack({give(out), give(fin)}) : give(out);
}

// ----------------------------------------------------------------------- beam

// (logits, scores, num_candidates or None, workspace) -> (scores, parents, tokens)
PyObject *beam_select(PyObject *const *a) {
  const Tensor &logits = tensor("logits", a[0]), &scores = tensor("scores", a[1]);
  const at::Device dev = logits.device();
  BAD_IF(!logits.is_cuda(), "logits must be a device tensor");
  BAD_IF(scores.device() != dev, "scores must be on ", dev);
  BAD_IF(logits.dim() != 3, "logits must be [batch, beams, vocabulary]");
  const int64_t B = logits.size(0), K = logits.size(1), V = logits.size(2);
  gdn_beam_params p{};
  p.logits_dtype = float_type(logits.scalar_type());
  BAD_IF(p.logits_dtype < 0, "logits must be float32, bfloat16 or float16");
  exactly("scores", scores, {B, K}, at::kFloat);
  no_derivative("logits", logits);
  no_derivative("scores", scores);
  BAD_IF(K < 1 || K > GDN_BEAM_MAX || V < 1 || V > (1 << 28) || B > INT32_MAX,
         "logits must have 1 to ", GDN_BEAM_MAX, " beams and 1 to 2^28 tokens");
  int64_t m = K;
  if (a[2] != Py_None) {
    m = PyLong_AsLongLong(a[2]);
    if (m == -1 && PyErr_Occurred()) throw PythonError{};
  }
  BAD_IF(m < 1 || m > GDN_BEAM_MAX || m > K * V, "num_candidates must be 1 to ", GDN_BEAM_MAX,
         " and at most beams x vocabulary");
  // beams at an even distance from each other, tokens side by side
  BAD_IF(V > 1 && logits.stride(2) != 1, "logits: the values of one beam must be contiguous");
  int64_t step = V;
  if (K > 1) step = logits.stride(1);
  else if (B > 1) step = logits.stride(0);
  BAD_IF(K > 1 && B > 1 && logits.stride(0) != K * step,
         "logits: all beams must be evenly spaced");
  BAD_IF(B * K > 1 && step < V, "logits must not overlap itself");
  p.num_groups = (int32_t)B;
  p.num_beams = (int32_t)K;
  p.vocab = (int32_t)V;
  p.num_candidates = (int32_t)m;
  p.logits = logits.data_ptr();
  p.logits_stride = step;
  p.scores = (const float *)scores.data_ptr();
  const Tensor best = fresh({B, m}, at::kFloat, dev), parents = fresh({B, m}, at::kInt, dev),
               tokens = fresh({B, m}, at::kInt, dev);
  p.out_scores = (float *)best.data_ptr();
  p.out_parents = (int32_t *)parents.data_ptr();
  p.out_tokens = (int32_t *)tokens.data_ptr();
  Tensor memory;
  p.workspace = workspace_for(a[3], lib.beam_workspace(&p), dev, memory, p.workspace_bytes);
  launch(dev, [&](void *s) { return lib.beam_select(&p, s); });
  return pack({give(best), give(parents), give(tokens)});
}

// (list of pools, state_indices, parents, output_indices, status) -> indices
PyObject *pool_reorder(PyObject *const *a) {
  const Py_ssize_t n = PyList_Check(a[0]) ? PyList_GET_SIZE(a[0]) : 0;
  BAD_IF(n < 1, "state_pool_reorder needs a pool");
  const Tensor &first = tensor("pool", PyList_GET_ITEM(a[0], 0));
  const at::Device dev = first.device();
  const Tensor &idx = row_list("state_indices", a[1], dev);
  const Tensor &parents = row_list("parents", a[2], dev);
  gdn_reorder_params p{};
  p.index_type = index_type("state_indices", idx);
  BAD_IF(parents.scalar_type() != idx.scalar_type() || parents.dim() != 2 ||
             !parents.is_contiguous(),
         "parents must be contiguous [batch, beams] of state_indices' dtype");
  BAD_IF(parents.numel() != idx.numel(), "state_indices must hold a row for each of the parents");
  BAD_IF(parents.size(1) < 1 || parents.size(1) > GDN_BEAM_MAX, "parents must have 1 to ",
         GDN_BEAM_MAX, " beams");
  const Tensor *out_ = optional("output_indices", a[3], dev);
  BAD_IF(out_ && (out_->scalar_type() != idx.scalar_type() || out_->sizes() != idx.sizes() ||
                  !out_->is_contiguous()),
         "output_indices must match state_indices");
  Writes writes;
  writes.add("output_indices", out_);
  p.status = (int32_t *)status_word(a[4], dev, writes);
  std::vector<gdn_reorder_pool> pools((size_t)n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const Tensor &pool = tensor("pool", PyList_GET_ITEM(a[0], i));
    BAD_IF(pool.device() != dev, "pools must share a device");
    writes.add("pool", pool);
    const PoolView v("pool", pool, true);
    BAD_IF(v.rows != first.size(0), "pools must share a number of rows");
    gdn_reorder_pool &q = pools[(size_t)i];
    q.pool = v.data;
    q.dtype = v.dtype;
    for (int k = 0; k < 3; ++k) q.extent[k] = v.extent[k];
    for (int k = 0; k < 4; ++k) q.strides[k] = v.strides[k];
  }
  p.num_groups = (int32_t)parents.size(0);
  p.num_beams = (int32_t)parents.size(1);
  p.num_pools = (int32_t)n;
  p.pool_rows = first.size(0);
  p.pools = pools.data();
  const Tensor out = out_ ? *out_ : fresh(idx.sizes(), idx.scalar_type(), dev);
  p.state_indices = idx.data_ptr();
  p.parents = parents.data_ptr();
  p.new_indices = out.data_ptr();
  launch(dev, [&](void *s) { return lib.pool_reorder(&p, s); });
  writes.done();
  return give(out);
}

}  // namespace calls
