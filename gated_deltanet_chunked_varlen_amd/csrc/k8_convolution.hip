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
// registers, so that each row is read once but for the W - 1 rows before a run.
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
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][e] = to_f32(p[e * W + j]);
      bias[e] = a.bias ? to_f32(((const Tw *)a.bias)[c + e]) : 0.f;
    }
  }
  static __device__ __forceinline__ const Tx *x_row(const ConvArgs &a, int64_t t, int c) {
    return (const Tx *)a.x + t * a.x_stride + c;
  }
  // x~ at place p of a sequence that starts at token bos (p < 0: its state,
  // state row r, zero without one)
  static __device__ __forceinline__ void seen(const ConvArgs &a, int bos, int p, int64_t r, int c,
                                              float (&o)[V]) {
    if (p >= 0) {
      widen(load_vec<Tx, V>(x_row(a, bos + p, c)), o);
    } else if (a.init.p && r >= 0) {
      state_read<V>(a.init, r * a.init.stride + (int64_t)(K + p) * a.C + c, o);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = 0.f;
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
  float w[W][V], bias[V], in[2 * K][V], end[K][V];
  F::taps(a, c, w, bias);
#pragma unroll
  for (int k = 0; k < 2 * K; ++k)
    if (k - K < len) F::seen(a, bos, k - K, r, c, in[k]);
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (a.fin.p) F::seen(a, bos, len - K + k, r, c, end[k]);
#pragma unroll
  for (int t = 0; t < K; ++t) {
    if (t >= len) break;
    float y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      y[e] = bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j) y[e] = fmaf(w[j][e], in[t + j][e], y[e]);
    }
    F::activate(a, y);
    store_vec<typename F::X, V>((typename F::X *)a.out + (int64_t)(bos + t) * a.C + c, y);
  }
  if (a.fin.p && r >= 0) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      state_write<V>(a.fin, r * a.fin.stride + (int64_t)k * a.C + c, end[k]);
  }
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
  float w[W][V], bias[V], in[2 * K][V], o[K][V];
  F::taps(a, c, w, bias);
#pragma unroll
  for (int k = 0; k < 2 * K; ++k)
    if (k - K < len) F::seen(a, bos, k - K, i, c, in[k]);
#pragma unroll
  for (int p = 0; p < K; ++p) {
#pragma unroll
    for (int e = 0; e < V; ++e) o[p][e] = 0.f;
    // x~ ends with its state's rows from len on
    if (a.dfin && p >= len)
      row_load<float, V>(a.dfin, ((int64_t)i * K + (p - len)) * a.C + c, o[p]);
  }
#pragma unroll
  for (int t = 0; t < K; ++t) {
    if (t >= len) break;
    float win[W][V], d[V];
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) win[j][e] = in[t + j][e];
    widen(load_vec<Tx, V>((const Tx *)a.dy + (int64_t)(bos + t) * a.dy_stride + c), d);
    token_gradient<F>(a, w, bias, win, d);
#pragma unroll
    for (int j = 0; t + j < K; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) o[t + j][e] = fmaf(w[j][e], d[e], o[t + j][e]);
  }
#pragma unroll
  for (int p = 0; p < K; ++p) row_store<float, V>(a.dinit, ((int64_t)i * K + p) * a.C + c, o[p]);
}

// One token of a run: the window moves on to token t (place pos of its
// sequence), d is formed and added to the open rows of dx.  `valid`: t belongs to
// a sequence; pos counts up to W at most.
template <typename F>
__device__ __forceinline__ void slide(const float (&x)[F::V], float (&win)[F::W][F::V]) {
#pragma unroll
  for (int j = 0; j + 1 < F::W; ++j)
#pragma unroll
    for (int e = 0; e < F::V; ++e) win[j][e] = win[j + 1][e];
#pragma unroll
  for (int e = 0; e < F::V; ++e) win[F::W - 1][e] = x[e];
}

template <typename Tx, typename Tw, int W, int V>
__global__ void __launch_bounds__(kThreads) conv_backward_kernel(ConvArgs a) {
  typedef ConvX<Tx, Tw, W, V> F;
  constexpr int K = W - 1, U = 4;
  __shared__ int mark[kThreads];
  __shared__ int pos_of[kThreads / 64][128], seq_of[kThreads / 64][128];
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
  // the run's tokens and the K behind it: bit s stands for token t0 + s
  typedef unsigned __int128 u128;
  u128 valid, last;
  {
    Block64 g = block_geometry(a.b, t0 - at, lane, mark + (threadIdx.x & ~63));
    pos_of[wave][lane] = g.pos;
    seq_of[wave][lane] = g.seq;
    valid = g.valid;
    last = g.last;
    g = block_geometry(a.b, t0 - at + 64, lane, mark + (threadIdx.x & ~63));
    pos_of[wave][64 + lane] = g.pos;
    seq_of[wave][64 + lane] = g.seq;
    valid |= (u128)g.valid << 64;
    last |= (u128)g.last << 64;
    valid >>= at;
    last >>= at;
  }
  wave_sync();
  if (c >= a.C) return;
  auto seq_at = [&](int s) { return __builtin_amdgcn_readfirstlane(seq_of[wave][at + s]); };
  auto pos_at = [&](int s) { return __builtin_amdgcn_readfirstlane(pos_of[wave][at + s]); };
  float w[W][V], bias[V], win[W][V], open[W][V], dw[W][V], db[V];
  F::taps(a, c, w, bias);
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) win[j][e] = open[j][e] = dw[j][e] = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) db[e] = 0.f;
  // rows before the run: win[1 ..] become the window's first ones
  if (valid & 1) {
    const int p = pos_at(0), i = seq_at(0);
#pragma unroll
    for (int j = 1; j < W; ++j)
      if (p > 0) F::seen(a, t0 - p, p - W + j, i, c, win[j]);
  }
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
  for (int s0 = 0; s0 < total; s0 += U) {
    Vec<Tx, V> nx[U], ny[U];
    if (s0 + U < total) fetch(s0 + U, nx, ny);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u;
      if (s < total) {
        float x[V];
        widen(rx[u], x);
        const bool here = (unsigned)(valid >> s) & 1;
        const int p = here ? pos_at(s) : 0;
        if (here && p == 0) {  // a sequence starts: the window holds its state
#pragma unroll
          for (int j = 1; j < W; ++j) F::seen(a, t0 + s, j - W, seq_at(s), c, win[j]);
        }
        slide<F>(x, win);
#pragma unroll
        for (int j = W - 1; j > 0; --j)
#pragma unroll
          for (int e = 0; e < V; ++e) open[j][e] = open[j - 1][e];
#pragma unroll
        for (int e = 0; e < V; ++e) open[0][e] = 0.f;
        if (here) {
          float d[V];
          widen(ry[u], d);
          token_gradient<F>(a, w, bias, win, d);
          // open[j]: dx of token t - j, which sees this token's d through tap W - 1 - j
#pragma unroll
          for (int j = 0; j < W; ++j)
            if (p >= j) {
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
          // the last K tokens of a sequence are its final state; where it ends
          // behind the last token looked at, the run's tokens are none of them
          if (a.dfin && ((unsigned)(last >> s) & 1)) {
            const int i = seq_at(s);
#pragma unroll
            for (int j = 0; j < K; ++j)
              if (p >= j) {
                float f[V];
                row_load<float, V>(a.dfin, ((int64_t)i * K + (K - 1 - j)) * a.C + c, f);
#pragma unroll
                for (int e = 0; e < V; ++e) open[j][e] += f[e];
              }
          }
        }
        const int t = t0 + s - K;
        if (s >= K && t <= end) store_vec<Tx, V>((Tx *)a.dx + (int64_t)t * a.C + c, open[K]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rx[u] = nx[u];
      ry[u] = ny[u];
    }
  }
  float *part = a.part + unit * (int64_t)(W + 1) * a.C + c;
#pragma unroll
  for (int j = 0; j < W; ++j) row_store<float, V>(part, (int64_t)j * a.C, dw[j]);
  row_store<float, V>(part, (int64_t)W * a.C, db);
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
    for (int r = part; r < a.parts; r += kParts) sum += a.part[r * n + id];
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
__global__ void __launch_bounds__(kThreads) conv_decode_kernel(ConvArgs a) {
  typedef ConvX<Tx, Tw, W, V> F;
  constexpr int K = W - 1;
  if (blockIdx.x == 0 && a.b.status) decode_status(a.b);
  const int per = (a.C + V - 1) / V;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= (int64_t)per * a.b.N) return;
  const int i = (int)(id / per), c = (int)(id % per) * V;
  const int64_t r = state_row(a.b, i);
  float w[W][V], bias[V], in[W][V], y[V];
#pragma unroll
  for (int j = 0; j < W; ++j) F::seen(a, i, j - K, r, c, in[j]);
  F::taps(a, c, w, bias);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    y[e] = bias[e];
#pragma unroll
    for (int j = 0; j < W; ++j) y[e] = fmaf(w[j][e], in[j][e], y[e]);
  }
  F::activate(a, y);
  store_vec<Tx, V>((Tx *)a.out + (int64_t)i * a.C + c, y);
  if (a.fin.p && r >= 0) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      state_write<V>(a.fin, r * a.fin.stride + (int64_t)k * a.C + c, in[k + 1]);
  }
}

template <template <typename, typename, int, int> class L, typename Tx, typename Tw>
hipError_t by_width(const ConvArgs &a, hipStream_t s) {
  constexpr int V = 16 / sizeof(Tx);
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
  static hipError_t go(const ConvArgs &a, hipStream_t s) {
    const unsigned grid = wave_grid(((int64_t)a.runs + a.b.N) * a.ncb);
    conv_forward_kernel<Tx, Tw, W, V><<<dim3(grid), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
  }
};
template <typename Tx, typename Tw, int W, int V> struct Bwd {
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
  static hipError_t go(const ConvArgs &a, hipStream_t s) {
    const int64_t threads = (int64_t)((a.C + V - 1) / V) * a.b.N;
    const unsigned grid = (unsigned)(threads > 0 ? (threads + kThreads - 1) / kThreads : 1);
    conv_decode_kernel<Tx, Tw, W, V><<<dim3(grid), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_conv_forward(const ConvArgs &a, hipStream_t s) { return dispatch<Fwd>(a, s); }
hipError_t launch_conv_backward(const ConvArgs &a, hipStream_t s) { return dispatch<Bwd>(a, s); }
hipError_t launch_conv_decode(const ConvArgs &a, hipStream_t s) { return dispatch<Dec>(a, s); }

}  // namespace gdn
