// k8_convolution.hip -- short causal depthwise convolution of packed sequences:
// forward, backward and decode step.
//
//     y_t = act(bias + sum_j w_j x~_{t + j}),   j < W
//
// where x~ is a sequence's state (its W - 1 last inputs from before) followed by
// its tokens, and the final state the last W - 1 rows of x~.
//
// Bounded by HBM: 2 W + a few operations per element of x.  A wave takes a run of
// tokens of 64 x V channels (V: 16 bytes of x) and slides the window along it in
// registers, so that each row is read once but for the W - 1 rows before a run
// (23 060 tokens of 8192 channels in bf16: 141 us, 5.4 TB/s, what a large copy
// reaches; their gradients, 300 us, 3.8 TB/s, with fp32 weights at three waves a SIMD,
// and a bound in most of its runs, as in 200 short sequences, 418 where 8 sequences
// took 281; a decode step of 256 sequences 9 us).
//
// Forward: tokens whose window lies inside their sequence need no state, and a
// run writes only those.  The first W - 1 tokens of a sequence and its final
// state are written by a wave of the sequence's own, which reads the state
// before it writes one: so a pool can be worked on in place in one launch.
#include "gdn_layers.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

template <typename Tx, typename Tw, int W_, int V_> struct Conv {
  static constexpr int W = W_, V = V_, K = W_ - 1;

  // w[j][e]: tap j of channel c + e (fp32)
  static __device__ __forceinline__ void taps(const ConvArgs &a, int c, float (&w)[W][V],
                                              float (&bias)[V]) {
    const Tw *p = (const Tw *)a.w + (int64_t)c * W;
    float o[V * W];
    if constexpr (V > 1) {
      widen(load_vec<Tw, V * W>(p), o);
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) o[j] = to_f32(p[j]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][e] = o[e * W + j];
      bias[e] = 0.f;
    }
    if (a.bias) widen(load_vec<Tw, V>((const Tw *)a.bias + c), bias);
  }
  static __device__ __forceinline__ const Tx *x_row(const ConvArgs &a, int64_t t, int c) {
    return (const Tx *)a.x + t * a.x_stride + c;
  }
  // the state of row r (zero without one)
  static __device__ __forceinline__ void state(const ConvArgs &a, int64_t r, int c,
                                               float (&o)[K][V]) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) o[k][e] = 0.f;
    if (!a.init.p || r < 0) return;
    int64_t off[K];
#pragma unroll
    for (int k = 0; k < K; ++k) off[k] = r * a.init.stride + (int64_t)k * a.C + c;
    state_read<K, V>(a.init, off, o);
  }
  static __device__ __forceinline__ void keep(const ConvArgs &a, int64_t r, int c,
                                              const float (&o)[K][V]) {
    int64_t off[K];
#pragma unroll
    for (int k = 0; k < K; ++k) off[k] = r * a.fin.stride + (int64_t)k * a.C + c;
    state_write<K, V>(a.fin, off, o);
  }
  // x~ at the K places from p on, those below `len`, of a sequence of which the
  // first row is token bos and the state `st` (others: unspecified)
  static __device__ __forceinline__ void seen(const ConvArgs &a, int bos, int len, int p, int c,
                                              const float (&st)[K][V], float (&o)[K][V]) {
    Vec<Tx, V> raw[K];
    if (len > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        raw[k] = load_vec<Tx, V>(x_row(a, bos + min(max(p + k, 0), len - 1), c));
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (len > 0 && p + k >= 0) {
        widen(raw[k], o[k]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) o[k][e] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (j == K + p + k) {
#pragma unroll
            for (int e = 0; e < V; ++e) o[k][e] = st[j][e];
          }
      }
    }
  }
  static __device__ __forceinline__ void activate(const ConvArgs &a, float (&o)[V]) {
    if (!a.silu) return;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] *= sigmoid(o[e]);
  }
  // d *= act'(pre)
  static __device__ __forceinline__ void chain(const ConvArgs &a, const float (&pre)[V],
                                               float (&d)[V]) {
    if (!a.silu) return;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float s = sigmoid(pre[e]);
      d[e] *= s * fmaf(pre[e], 1.f - s, 1.f);
    }
  }
};

// Wave-uniform place of a wave in the grid: run or sequence, and channel.
__device__ __forceinline__ int64_t wave_id() {
  return (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// The first W - 1 tokens of sequence i and its final state.
template <typename F>
__device__ __forceinline__ void forward_sequence(const ConvArgs &a, int i, int c, int lane) {
  constexpr int W = F::W, V = F::V, K = F::K;
  int bos, len;
  sequence_of(a.b, i, lane, bos, len);
  if (c >= a.C) return;
  const int64_t r = state_row(a.b, i);
  float w[W][V], bias[V], st[K][V], x[K][V], end[K][V];
  F::taps(a, c, w, bias);
  F::state(a, r, c, st);
  F::seen(a, bos, len, 0, c, st, x);
  F::seen(a, bos, len, len - K, c, st, end);
#pragma unroll
  for (int t = 0; t < K; ++t) {
    if (t >= len) break;
    float y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      y[e] = bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j) y[e] = fmaf(w[j][e], t + j < K ? st[t + j][e] : x[t + j - K][e], y[e]);
    }
    F::activate(a, y);
    store_vec<typename F::X, V>((typename F::X *)a.out + (int64_t)(bos + t) * a.C + c, y);
  }
  if (a.fin.p && r >= 0) F::keep(a, r, c, end);
}

template <typename Tx, typename Tw, int W, int V>
struct ConvX : Conv<Tx, Tw, W, V> {
  typedef Tx X;
};

// Waves: the runs of tokens, channel blocks fastest, then the sequences.
template <typename Tx, typename Tw, int W, int V>
__global__ void __launch_bounds__(kThreads) conv_forward_kernel(ConvArgs a) {
  typedef ConvX<Tx, Tw, W, V> F;
  constexpr int K = W - 1, U = 4;  // tokens under way
  __shared__ int mark[kThreads];
  const int lane = threadIdx.x & 63;
  if (blockIdx.x == 0 && threadIdx.x < 64 && a.b.status && !a.b.bos) batch_status(a.b, lane);
  const int64_t id = wave_id();
  const int64_t unit = id / a.ncb;
  const int c = ((int)(id % a.ncb) * 64 + lane) * V;
  if (unit >= a.runs) {
    if (unit - a.runs < a.b.N) forward_sequence<F>(a, (int)(unit - a.runs), c, lane);
    return;
  }
  const int t0 = (int)unit * a.run, at = t0 & 63;
  const Block64 g = block_geometry(a.b, t0 - at, lane, mark + (threadIdx.x & ~63));
  unsigned long long todo = __ballot((g.valid >> lane & 1) && g.pos >= K) >> at;
  if (a.run < 64) todo &= (1ull << a.run) - 1;
  if (todo == 0 || c >= a.C) return;
  float w[W][V], bias[V], win[K][V];
  F::taps(a, c, w, bias);
#pragma unroll
  for (int k = 0; k < K; ++k) widen(load_vec<Tx, V>(F::x_row(a, max(t0 - K + k, 0), c)), win[k]);
  const int end = (int)a.b.T - 1;
  Vec<Tx, V> raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u] = load_vec<Tx, V>(F::x_row(a, min(t0 + u, end), c));
  for (int s = 0; s < a.run; s += U) {
    Vec<Tx, V> next[U];
    if (s + U < a.run) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        next[u] = load_vec<Tx, V>(F::x_row(a, min(t0 + s + U + u, end), c));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[V], y[V];
      widen(raw[u], x);
      if (todo >> (s + u) & 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          y[e] = fmaf(w[0][e], win[0][e], bias[e]);
#pragma unroll
          for (int j = 1; j < K; ++j) y[e] = fmaf(w[j][e], win[j][e], y[e]);
          y[e] = fmaf(w[K][e], x[e], y[e]);
        }
        F::activate(a, y);
        store_vec<Tx, V>((Tx *)a.out + (int64_t)(t0 + s + u) * a.C + c, y);
      }
#pragma unroll
      for (int k = 0; k + 1 < K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) win[k][e] = win[k + 1][e];
#pragma unroll
      for (int e = 0; e < V; ++e) win[K - 1][e] = x[e];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = next[u];
  }
}

// ------------------------------------------------------------------ backward
//
// With d_t = dy_t act'(pre_t), pre formed again from x:
//     dx~_p = sum_j w_j d_{p - j} (+ dfinal where x~ ends)
//     dw_j = sum_t d_t x~_{t + j},   dbias = sum_t d_t
// A run slides along x and dy, W - 1 tokens further than its own, and holds the
// W rows of dx that are open in registers.  dw and dbias are summed over the
// run in registers and stored; a second kernel adds the runs.  Gradients of
// initial states, which see the first W - 1 tokens only, are a wave of the
// sequence's own.

// d of a token from its window.
template <typename F>
__device__ __forceinline__ void token_gradient(const ConvArgs &a, const float (&w)[F::W][F::V],
                                               const float (&bias)[F::V],
                                               const float (&win)[F::W][F::V],
                                               float (&d)[F::V]) {
  float pre[F::V];
#pragma unroll
  for (int e = 0; e < F::V; ++e) {
    pre[e] = bias[e];
#pragma unroll
    for (int j = 0; j < F::W; ++j) pre[e] = fmaf(w[j][e], win[j][e], pre[e]);
  }
  F::chain(a, pre, d);
}

template <typename F>
__device__ __forceinline__ void backward_sequence(const ConvArgs &a, int i, int c, int lane) {
  constexpr int W = F::W, V = F::V, K = F::K;
  typedef typename F::X Tx;
  int bos, len;
  sequence_of(a.b, i, lane, bos, len);
  if (c >= a.C) return;
  float w[W][V], bias[V], st[K][V], x[K][V], o[K][V];
  F::taps(a, c, w, bias);
  F::state(a, i, c, st);
  F::seen(a, bos, len, 0, c, st, x);
#pragma unroll
  for (int p = 0; p < K; ++p) {
#pragma unroll
    for (int e = 0; e < V; ++e) o[p][e] = 0.f;
    // x~ ends with its state's rows from len on
    if (a.dfin && p >= len)
      f32_load<V>(a.dfin + ((int64_t)i * K + (p - len)) * a.C + c, a.fvec, o[p]);
  }
#pragma unroll
  for (int t = 0; t < K; ++t) {
    if (t >= len) break;
    float win[W][V], d[V];
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) win[j][e] = t + j < K ? st[t + j][e] : x[t + j - K][e];
    widen(load_vec<Tx, V>((const Tx *)a.dy + (int64_t)(bos + t) * a.dy_stride + c), d);
    token_gradient<F>(a, w, bias, win, d);
#pragma unroll
    for (int j = 0; t + j < K; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) o[t + j][e] = fmaf(w[j][e], d[e], o[t + j][e]);
  }
  int64_t off[K];
#pragma unroll
  for (int p = 0; p < K; ++p) off[p] = ((int64_t)i * K + p) * a.C + c;
  rows_store<float, K, V>(a.dinit, a.fvec, off, o);
}

// The window moves on by one token.
template <typename F>
__device__ __forceinline__ void slide(const float (&x)[F::V], float (&win)[F::W][F::V]) {
#pragma unroll
  for (int j = 0; j + 1 < F::W; ++j)
#pragma unroll
    for (int e = 0; e < F::V; ++e) win[j][e] = win[j + 1][e];
#pragma unroll
  for (int e = 0; e < F::V; ++e) win[F::W - 1][e] = x[e];
}

// Marks of a run's tokens and the K behind it: bit s stands for token t0 + s.
struct RunMarks {
  typedef unsigned __int128 u128;
  u128 valid, first, last;
  int place;       // of the run's first token in its sequence
  const int *seq;  // of the run's tokens, in LDS
  __device__ __forceinline__ bool at(u128 m, int s) const { return (unsigned)(m >> s) & 1; }
  __device__ __forceinline__ int seq_at(int s) const {
    return __builtin_amdgcn_readfirstlane(seq[s]);
  }
};

// One run.  PLAIN: its tokens and the K before and behind it lie in the middle of
// one sequence, U tokens are under way.  Else one token after the other: whatever
// a bound takes (states, marks) would cost the plain runs their registers.
template <typename F, bool PLAIN>
__device__ __forceinline__ void backward_run(const ConvArgs &a, const RunMarks &m, int t0, int c,
                                             int64_t unit) {
  constexpr int W = F::W, V = F::V, K = F::K, U = PLAIN ? 4 : 1;
  typedef typename F::X Tx;
  float w[W][V], bias[V], win[W][V], open[W][V], dw[W][V], db[V];
  F::taps(a, c, w, bias);
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) win[j][e] = open[j][e] = dw[j][e] = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) db[e] = 0.f;
  const int end = (int)a.b.T - 1, total = a.run + K;
  Vec<Tx, V> rx[U], ry[U];
  auto fetch = [&](int s, Vec<Tx, V>(&vx)[U], Vec<Tx, V>(&vy)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = min(t0 + s + u, end);
      vx[u] = load_vec<Tx, V>(F::x_row(a, t, c));
      vy[u] = load_vec<Tx, V>((const Tx *)a.dy + (int64_t)t * a.dy_stride + c);
    }
  };
  fetch(0, rx, ry);
  if (PLAIN) {
#pragma unroll
    for (int j = 1; j < W; ++j) widen(load_vec<Tx, V>(F::x_row(a, t0 - W + j, c)), win[j]);
  }
#pragma unroll 1
  for (int s0 = 0; s0 < total; s0 += U) {
    Vec<Tx, V> nx[U], ny[U];
    if (s0 + U < total) fetch(s0 + U, nx, ny);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u;
      if (s >= total) break;
      // a new open row: open[j] is dx of token s - j, which sees this token's d
      // through tap W - 1 - j
#pragma unroll
      for (int j = W - 1; j > 0; --j)
#pragma unroll
        for (int e = 0; e < V; ++e) open[j][e] = open[j - 1][e];
#pragma unroll
      for (int e = 0; e < V; ++e) open[0][e] = 0.f;
      if (PLAIN || m.at(m.valid, s)) {
        int sees = K;  // tokens back to the run's first one, or its sequence's
        if (!PLAIN) {
          sees = s;
#pragma unroll
          for (int j = K; j >= 0; --j)
            if (s >= j && m.at(m.first, s - j)) sees = j;
          const bool starts = m.at(m.first, s);
          if (starts || s == 0) {  // the rows that the window moves on from
            const int p = starts ? 0 : m.place;
            float st[K][V], o[K][V];
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
              for (int e = 0; e < V; ++e) st[k][e] = 0.f;
            if (p < K) F::state(a, m.seq_at(s), c, st);
            F::seen(a, t0 + s - p, p, p - K, c, st, o);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
              for (int e = 0; e < V; ++e) win[k + 1][e] = o[k][e];
          }
        }
        float x[V], d[V];
        widen(rx[u], x);
        widen(ry[u], d);
        slide<F>(x, win);
        token_gradient<F>(a, w, bias, win, d);
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (PLAIN || sees >= j) {
#pragma unroll
            for (int e = 0; e < V; ++e) open[j][e] = fmaf(w[W - 1 - j][e], d[e], open[j][e]);
          }
        if (s < a.run) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            db[e] += d[e];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][e] = fmaf(d[e], win[j][e], dw[j][e]);
          }
        }
        // the last K tokens of a sequence are its final state (of one that ends
        // behind the last token looked at, they are not the run's)
        if (!PLAIN && a.dfin && m.at(m.last, s)) {
          const int64_t from = (int64_t)m.seq_at(s) * K;
#pragma unroll
          for (int j = 0; j < K; ++j)
            if (sees >= j) {
              float f[V];
              f32_load<V>(a.dfin + (from + (K - 1 - j)) * a.C + c, a.fvec, f);
#pragma unroll
              for (int e = 0; e < V; ++e) open[j][e] += f[e];
            }
        }
      }
      const int t = t0 + s - K;
      if (s >= K && t <= end) store_vec<Tx, V>((Tx *)a.dx + (int64_t)t * a.C + c, open[K]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rx[u] = nx[u];
      ry[u] = ny[u];
    }
  }
  int64_t off[W];
  float *part = a.part + unit * (int64_t)(W + 1) * a.C;
#pragma unroll
  for (int j = 0; j < W; ++j) off[j] = (int64_t)j * a.C + c;
  rows_store<float, W, V>(part, a.fvec, off, dw);
  const int64_t behind[1] = {(int64_t)W * a.C + c};
  const float(&sum)[1][V] = reinterpret_cast<const float(&)[1][V]>(db);
  rows_store<float, 1, V>(part, a.fvec, behind, sum);
}

template <typename Tx, typename Tw, int W, int V>
__global__ void __launch_bounds__(kThreads, 3) conv_backward_kernel(ConvArgs a) {
  typedef ConvX<Tx, Tw, W, V> F;
  typedef RunMarks::u128 u128;
  constexpr int K = W - 1;
  __shared__ int mark[kThreads];
  __shared__ int seq_of[kThreads / 64][128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x == 0 && threadIdx.x < 64 && a.b.status && !a.b.bos) batch_status(a.b, lane);
  const int64_t id = wave_id();
  const int64_t unit = id / a.ncb;
  const int c = ((int)(id % a.ncb) * 64 + lane) * V;
  if (unit >= a.runs) {
    if (a.dinit && unit - a.runs < a.b.N) backward_sequence<F>(a, (int)(unit - a.runs), c, lane);
    return;
  }
  const int t0 = (int)unit * a.run, at = t0 & 63;
  RunMarks m;
  Block64 g = block_geometry(a.b, t0 - at, lane, mark + (threadIdx.x & ~63));
  seq_of[wave][lane] = g.seq;
  m.valid = g.valid;
  m.first = g.first;
  m.last = g.last;
  m.place = __builtin_amdgcn_readlane(g.pos, at);
  g = block_geometry(a.b, t0 - at + 64, lane, mark + (threadIdx.x & ~63));
  seq_of[wave][64 + lane] = g.seq;
  m.valid = (m.valid | (u128)g.valid << 64) >> at;
  m.first = (m.first | (u128)g.first << 64) >> at;
  m.last = (m.last | (u128)g.last << 64) >> at;
  m.seq = seq_of[wave] + at;
  wave_sync();
  if (c >= a.C) return;
  const u128 all = ((u128)1 << (a.run + K)) - 1;
  const bool plain = (m.valid & all) == all && (m.first & all) == 0 && (m.last & all) == 0 &&
                     m.place >= K;
  if (plain) backward_run<F, true>(a, m, t0, c, unit);
  else backward_run<F, false>(a, m, t0, c, unit);
}

// dw and dbias: the runs' sums, added in the order of the runs by eight threads
// a column (and then over these).
template <int W> __global__ void __launch_bounds__(kThreads) conv_sums_kernel(ConvArgs a) {
  constexpr int kCols = 32, kParts = kThreads / kCols;
  __shared__ float sums[kParts][kCols];
  const int col = threadIdx.x % kCols, part = threadIdx.x / kCols;
  const int64_t id = (int64_t)blockIdx.x * kCols + col, n = (int64_t)(W + 1) * a.C;
  float sum = 0.f;
  if (id < n) {
#pragma unroll 4
    for (int r = part; r < a.runs; r += kParts) sum += a.part[r * n + id];
  }
  sums[part][col] = sum;
  __syncthreads();
  if (part != 0 || id >= n) return;
#pragma unroll
  for (int p = 1; p < kParts; ++p) sum += sums[p][col];
  const int j = (int)(id / a.C), c = (int)(id % a.C);
  if (j < W) a.dw[(int64_t)c * W + j] = sum;
  else if (a.db) a.db[c] = sum;
}

// -------------------------------------------------------------------- decode

// One thread per V channels of a sequence: reads its state and its token, writes
// the output and the state moved on by one.
template <typename Tx, typename Tw, int W, int V>
__global__ void __launch_bounds__(kThreads) conv_decode_kernel(ConvArgs a, int blocks) {
  typedef ConvX<Tx, Tw, W, V> F;
  constexpr int K = W - 1;
  if (blockIdx.x == 0 && a.b.status) decode_status(a.b);
  const int i = blockIdx.x / blocks;
  const int c = ((int)(blockIdx.x % blocks) * kThreads + threadIdx.x) * V;
  if (i >= a.b.N || c >= a.C) return;
  const int64_t r = state_row(a.b, i);
  float w[W][V], bias[V], st[K][V], x[V], y[V];
  const Vec<Tx, V> raw = load_vec<Tx, V>(F::x_row(a, i, c));
  F::taps(a, c, w, bias);
  F::state(a, r, c, st);
  widen(raw, x);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    y[e] = bias[e];
#pragma unroll
    for (int j = 0; j < W; ++j) y[e] = fmaf(w[j][e], j < K ? st[j][e] : x[e], y[e]);
  }
  F::activate(a, y);
  store_vec<Tx, V>((Tx *)a.out + (int64_t)i * a.C + c, y);
  if (!a.fin.p || r < 0) return;
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) st[k][e] = st[k + 1][e];
    st[K - 1][e] = x[e];
  }
  F::keep(a, r, c, st);
}

template <template <typename, typename, int, int> class L, typename Tx, typename Tw>
hipError_t by_width(const ConvArgs &a, hipStream_t s) {
  constexpr int V = conv_lane(L<Tx, Tw, 2, 1>::kMode, (int)sizeof(Tx));
  if (a.W == 2) return a.vec ? L<Tx, Tw, 2, V>::go(a, s) : L<Tx, Tw, 2, 1>::go(a, s);
  if (a.W == 3) return a.vec ? L<Tx, Tw, 3, V>::go(a, s) : L<Tx, Tw, 3, 1>::go(a, s);
  return a.vec ? L<Tx, Tw, 4, V>::go(a, s) : L<Tx, Tw, 4, 1>::go(a, s);
}
template <template <typename, typename, int, int> class L>
hipError_t dispatch(const ConvArgs &a, hipStream_t s) {
  if (a.x_dtype == GDN_F32) return by_width<L, float, float>(a, s);
  if (a.x_dtype == GDN_BF16)
    return a.w_dtype == GDN_F32 ? by_width<L, bf16, float>(a, s) : by_width<L, bf16, bf16>(a, s);
  return a.w_dtype == GDN_F32 ? by_width<L, f16, float>(a, s) : by_width<L, f16, f16>(a, s);
}

unsigned wave_grid(int64_t waves) {
  const int64_t per = kThreads / 64;
  return (unsigned)(waves > 0 ? (waves + per - 1) / per : 1);
}

template <typename Tx, typename Tw, int W, int V> struct Fwd {
  static constexpr int kMode = 0;
  static hipError_t go(const ConvArgs &a, hipStream_t s) {
    const unsigned grid = wave_grid(((int64_t)a.runs + a.b.N) * a.ncb);
    conv_forward_kernel<Tx, Tw, W, V><<<dim3(grid), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
  }
};
template <typename Tx, typename Tw, int W, int V> struct Bwd {
  static constexpr int kMode = 1;
  static hipError_t go(const ConvArgs &a, hipStream_t s) {
    const unsigned grid = wave_grid(((int64_t)a.runs + (a.dinit ? a.b.N : 0)) * a.ncb);
    conv_backward_kernel<Tx, Tw, W, V><<<dim3(grid), dim3(kThreads), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t cols = (int64_t)(W + 1) * a.C;
    conv_sums_kernel<W><<<dim3((unsigned)((cols + 31) / 32)), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
  }
};
template <typename Tx, typename Tw, int W, int V> struct Dec {
  static constexpr int kMode = 2;
  static hipError_t go(const ConvArgs &a, hipStream_t s) {
    const int blocks = (a.C + kThreads * V - 1) / (kThreads * V);
    const int64_t n = a.b.N > 0 ? a.b.N : 1;
    conv_decode_kernel<Tx, Tw, W, V>
        <<<dim3((unsigned)(blocks * n)), dim3(kThreads), 0, s>>>(a, blocks);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_conv_forward(const ConvArgs &a, hipStream_t s) { return dispatch<Fwd>(a, s); }
hipError_t launch_conv_backward(const ConvArgs &a, hipStream_t s) { return dispatch<Bwd>(a, s); }
hipError_t launch_conv_decode(const ConvArgs &a, hipStream_t s) { return dispatch<Dec>(a, s); }

}  // namespace gdn
