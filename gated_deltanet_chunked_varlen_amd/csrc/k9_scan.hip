// k9_scan.hip -- selective state space scan of packed sequences: forward pass over
// tiles and decode step (k10_scan_backward.hip: backward pass; k12_scan_walk.hip: the
// forward pass of batches that take less than that).
//
// With step size d_t = softplus(delta_t + delta_bias) (or as given), for every
// channel c and each of its N states n, in fp32,
//     h_t = exp(d_t A) h_{t-1} + d_t B_t x_t
//     y_t = sum_n C_t h_t + D x_t,     output_t = y_t silu(z_t)
//
// Bounded by the vector ALU: a token takes, for each state, the exponential (the
// cost of two other operations), its argument, the input's product and two
// fused products, 24 cycles of a SIMD per 64 states, against 8 bytes of a
// channel's token for all of its states (16384 tokens of 4096 channels with 16
// states: 164 us of such work, 104 us of memory; the passes take 803 us, as they
// form the states twice and their waves wait for the scalar loads).  So a lane holds one channel with all of
// its states in registers, B and C (the same for all channels of a group) come
// through scalar registers, and nothing crosses lanes.
//
// Time is cut into tiles of L tokens, and a pass over tiles takes three kernels:
//   states   every tile's own last state from zero, and the sum of its step
//            sizes, which is all that a state's way across a tile depends on
//            (exp(A sum d) is the product of the decays)
//   chain    the state before each tile, tile after tile, per channel and state
//   forward  the tiles again from there, with outputs
// Where one tile holds all tokens the last kernel is the only one.
//
// Sequence bounds.  Where a sequence starts the state is replaced by its
// initial state, never multiplied by zero.  A sequence's initial state is read
// by the tile where it starts, in the first kernel; if the sequence goes on
// into later tiles it is kept in the workspace, as the last kernel may have
// written its final state over it in a pool worked on in place.  A decay over a
// tile that underflows is kept at the smallest number above 0, so that an
// infinite state stays infinite.
#include "gdn_scan.h"

#include <algorithm>
#include <type_traits>

#pragma clang fp contract(off)

namespace gdn {

using namespace scan;

namespace {

// ------------------------------------------------------------------- prepare

// B and C in fp32, padded with zeros: by token (scan and chain) and, for the
// backward pass, by state; log2(e) A by state.
template <typename Tx>
__global__ void __launch_bounds__(kThreads) scan_prepare_kernel(ScanArgs a, int ns) {
  const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  const int64_t per = 2 * (int64_t)ns, n = a.b.T * a.G * per;
  auto value = [&](int64_t t, int g, int which, int k) {
    if (k >= a.N || t >= a.b.T) return 0.f;
    const Tx *p = which ? (const Tx *)a.C_ + t * a.c_stride : (const Tx *)a.B + t * a.b_stride;
    return to_f32(p[(int64_t)g * a.N + k]);
  };
  for (int64_t i = at; i < n; i += step) {
    const int64_t row = i / per;
    const int k = (int)(i % per);
    a.bc[i] = value(row / a.G, (int)(row % a.G), k / ns, k % ns);
  }
  if (a.bct) {
    const int64_t m = a.G * per * a.Tp;
    for (int64_t i = at; i < m; i += step) {
      const int64_t row = i / a.Tp;
      a.bct[i] = value(i % a.Tp, (int)(row / per), (int)(row % per) / ns, (int)(row % ns));
    }
  }
  const int64_t m = (int64_t)ns * a.C;
  for (int64_t i = at; i < m; i += step) {
    const int k = (int)(i / a.C), c = (int)(i % a.C);
    a.a2[i] = k < a.N ? kLog2E * a.A[(int64_t)c * a.N + k] : 0.f;
  }
}

// ------------------------------------------------------------------- forward

// `count` states of a lane's channel, into and from LDS (state n of lane l at
// n * 64 + l; `lds` is the lane's first).
template <typename St>
__device__ __forceinline__ void stage_in(const StateRows &s, int64_t off, int count, float *lds) {
#pragma unroll 4
  for (int n = 0; n < count; ++n) lds[n * 64] = to_f32(((const St *)s.p)[off + n]);
}
template <typename St>
__device__ __forceinline__ void stage_out(const StateRows &s, int64_t off, int count,
                                          const float *lds) {
#pragma unroll 4
  for (int n = 0; n < count; ++n) ((St *)s.p)[off + n] = from_f32<St>(lds[n * 64]);
}

// Whether a lane's states are whole aligned vectors of fp32.
template <int NS>
__device__ __forceinline__ bool plain_rows(const StateRows &s, int count) {
  return s.dtype == GDN_F32 && count == NS && s.stride % 4 == 0 && ((uintptr_t)s.p & 15) == 0;
}

// States of sequence i, channel c, before its first token and behind its last.
// Rows of other types and lengths go through LDS, one state after the other:
// unrolled they would take the registers that the scan is to use.
template <int NS>
__device__ __forceinline__ void initial_state(const ScanArgs &a, int i, int c, float *lds,
                                              float (&h)[NS]) {
#pragma unroll
  for (int n = 0; n < NS; ++n) h[n] = 0.f;
  const int64_t r = a.init.p ? state_row(a.b, i) : -1;
  if (r < 0) return;
  const int64_t off = r * a.init.stride + (int64_t)c * a.N;
  if (plain_rows<NS>(a.init, a.N)) {
    const f32x4 *p = (const f32x4 *)((const float *)a.init.p + off);
#pragma unroll
    for (int n = 0; n < NS; n += 4) {
      const f32x4 v = p[n / 4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[n + e] = v[e];
    }
    return;
  }
  if (a.init.dtype == GDN_F32) stage_in<float>(a.init, off, a.N, lds);
  else if (a.init.dtype == GDN_BF16) stage_in<bf16>(a.init, off, a.N, lds);
  else if (a.init.dtype == GDN_F16) stage_in<f16>(a.init, off, a.N, lds);
  else if (a.init.dtype == GDN_FP8_E4M3) stage_in<fp8e4m3>(a.init, off, a.N, lds);
  else stage_in<fp8e5m2>(a.init, off, a.N, lds);
#pragma unroll
  for (int n = 0; n < NS; ++n)
    if (n < a.N) h[n] = lds[n * 64];
}
template <int NS>
__device__ __forceinline__ void final_state(const ScanArgs &a, int i, int c, float *lds,
                                            const float (&h)[NS]) {
  const int64_t r = state_row(a.b, i);
  if (r < 0) return;
  const int64_t off = r * a.fin.stride + (int64_t)c * a.N;
  if (plain_rows<NS>(a.fin, a.N)) {
    f32x4 *p = (f32x4 *)((float *)a.fin.p + off);
#pragma unroll
    for (int n = 0; n < NS; n += 4) p[n / 4] = f32x4{h[n], h[n + 1], h[n + 2], h[n + 3]};
    return;
  }
#pragma unroll
  for (int n = 0; n < NS; ++n) lds[n * 64] = h[n];
  if (a.fin.dtype == GDN_F32) stage_out<float>(a.fin, off, a.N, lds);
  else if (a.fin.dtype == GDN_BF16) stage_out<bf16>(a.fin, off, a.N, lds);
  else if (a.fin.dtype == GDN_F16) stage_out<f16>(a.fin, off, a.N, lds);
  else if (a.fin.dtype == GDN_FP8_E4M3) stage_out<fp8e4m3>(a.fin, off, a.N, lds);
  else stage_out<fp8e5m2>(a.fin, off, a.N, lds);
}

// Final states of the empty sequences, by workgroups behind the tiles': their
// initial states.  A row of workgroups (`slice` of `slices`) takes every
// a.empties-th sequence.
__device__ __forceinline__ void empty_sequences(const ScanArgs &a, int part, int slice,
                                                int slices) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)a.C * a.N, step = (int64_t)slices * kThreads;
  for (int i = part; i < a.b.N; i += a.empties) {
    int bos, len;
    sequence_of(a.b, i, lane, bos, len);
    const int64_t r = state_row(a.b, i);
    if (len != 0 || r < 0) continue;
    for (int64_t e = slice * kThreads + threadIdx.x; e < row; e += U * step) {
      int64_t from[U], to[U];
      float v[U][1];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = min(e + u * step, row - 1);
        from[u] = r * a.init.stride + at;
        to[u] = r * a.fin.stride + at;
        v[u][0] = 0.f;
      }
      if (a.init.p) state_read<U, 1>(a.init, from, v);
      state_write<U, 1>(a.fin, to, v);
    }
  }
}

// OUT false: a tile's own last state, the sum of its step sizes, and the initial
// state of a sequence that starts in it and goes on.  OUT true: outputs and
// final states from the state before the tile.  FULL: N = NS.
template <typename Tx, int NS, bool OUT, bool FULL>
__global__ void __launch_bounds__(kThreads, scan_waves(NS)) scan_tile_kernel(ScanArgs a) {
  __shared__ TileGeo G;
  __shared__ float s_states[kWaves][NS][64], s_run[kWaves][3 * kRun][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ncw = (a.ncb + kWaves - 1) / kWaves;
  const int tile = blockIdx.x / ncw;
  // the first kernel of a call writes the status word
  if (blockIdx.x == 0 && wave == 0 && a.b.status && !a.b.bos && (!OUT || a.ntiles <= 1))
    batch_status(a.b, lane);
  if (tile >= a.ntiles) {
    if (OUT && tile - a.ntiles < a.empties)
      empty_sequences(a, tile - a.ntiles, blockIdx.x % ncw, ncw);
    return;
  }
  const int t0 = tile * a.L;
  tile_geometry(a, t0, G);
  const int cb = (int)(blockIdx.x % ncw) * kWaves + wave;
  if (cb >= a.ncb) return;
  float *const lds = &s_states[wave][0][lane], *const run = &s_run[wave][0][lane];
  const Channel ch(a, cb, lane);
  const int c = ch.c, end = (int)a.b.T - 1;
  float A2[NS], h[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) A2[n] = *lane_of<float>(a.a2, (int64_t)n * a.C, (unsigned)c * 4);
  const int64_t row = (int64_t)tile * a.N * a.C;
  const unsigned c4 = (unsigned)c * 4;
#pragma unroll
  for (int n = 0; n < NS; ++n)
    h[n] = OUT && a.ntiles > 1 && n < a.N ? *lane_of<float>(a.chunk, row + (int64_t)n * a.C, c4) : 0.f;
  const float bias = a.dbias ? a.dbias[c] : 0.f, D = OUT && a.D ? a.D[c] : 0.f;
  const float *bc = a.bc + (int64_t)ch.g * 2 * NS;
  const int64_t bcs = (int64_t)a.G * 2 * NS;
  float span = 0.f;
  Rows<Tx, kRun> rx, rd, rz;
  rx.load(a.x, a.x_stride, t0, end, c);
  rd.load(a.delta, a.delta_stride, t0, end, c);
  if (OUT && a.z) rz.load(a.z, a.z_stride, t0, end, c);
  const int L = min(a.L, (int)a.b.T - t0);
  for (int s = 0; s < L; s += kRun) {
    const int t = t0 + s;
    const Marks m(G, (t0 & 63) + s, kRun);
    float x[kRun], dt[kRun], z[kRun];
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      x[u] = to_f32(rx.v[u]);
      dt[u] = step_size(a, to_f32(rd.v[u]) + bias);
      z[u] = OUT && a.z ? to_f32(rz.v[u]) : 0.f;
    }
    if (s + kRun < L) {
      rx.load(a.x, a.x_stride, t + kRun, end, c);
      rd.load(a.delta, a.delta_stride, t + kRun, end, c);
      if (OUT && a.z) rz.load(a.z, a.z_stride, t + kRun, end, c);
    }
    char *const orow = uniform((char *)a.out + (int64_t)t * a.C * (int)sizeof(Tx));
    auto token = [&](int u, float x, float dt, float z) {
      float y = OUT ? skip_of(a, D, x) : 0.f;
      token_step<NS, OUT, FULL>(bc + (t + u) * bcs, dt, dt * x, A2, h, y, a.N);
      if (OUT) {
        if (a.z) y *= z * sigmoid(z);
        if (ch.ok)
          *(Tx *)(orow + (int64_t)u * a.C * (int)sizeof(Tx) + (unsigned)c * (unsigned)sizeof(Tx)) =
              from_f32<Tx>(y);
      } else {
        span += dt;
      }
    };
    if (m.valid == (1u << kRun) - 1 && (m.first | m.last) == 0) {
#pragma unroll
      for (int u = 0; u < kRun; ++u) token(u, x[u], dt[u], z[u]);
      continue;
    }
    // a sequence starts or ends here: one token after the other, by way of LDS
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      run[u * 64] = x[u];
      run[(kRun + u) * 64] = dt[u];
      if (OUT) run[(2 * kRun + u) * 64] = z[u];
    }
#pragma unroll 1
    for (int u = 0; u < kRun; ++u) {
      if (!(m.valid >> u & 1)) continue;
      if (m.first >> u & 1) {
        const int i = m.seq_at(u);
        // a sequence that goes on into the next tile: the last one of this tile
        const bool stays = a.ntiles > 1 && m.seq_at(u) == __builtin_amdgcn_readfirstlane(
                               G.seq[(t0 & 63) + L - 1]) &&
                           !(bits_at(G.last, (t0 & 63) + L - 1, 1));
        if (OUT && stays) {
#pragma unroll 1
          for (int n = 0; n < a.N; ++n)
            lds[n * 64] = *lane_of<float>(a.start, row + (int64_t)n * a.C, c4);
#pragma unroll
          for (int n = 0; n < NS; ++n) h[n] = n < a.N ? lds[n * 64] : 0.f;
        } else {
          initial_state<NS>(a, i, c, lds, h);
        }
        if (!OUT && stays && ch.ok) {
#pragma unroll
          for (int n = 0; n < NS; ++n) lds[n * 64] = h[n];
#pragma unroll 1
          for (int n = 0; n < a.N; ++n)
            *lane_of<float>(a.start, row + (int64_t)n * a.C, c4) = lds[n * 64];
        }
        span = 0.f;
      }
      token(u, run[u * 64], run[(kRun + u) * 64], OUT ? run[(2 * kRun + u) * 64] : 0.f);
      if (OUT && a.fin.p && ch.ok && (m.last >> u & 1)) final_state<NS>(a, m.seq_at(u), c, lds, h);
    }
  }
  if (!ch.ok) return;
  if (OUT) {  // of a single tile the state before it, which the caller may keep
    if (a.ntiles == 1 && a.chunk)
      for (int n = 0; n < a.N; ++n) *lane_of<float>(a.chunk, row + (int64_t)n * a.C, c4) = 0.f;
    return;
  }
#pragma unroll
  for (int n = 0; n < NS; ++n)
    if (n < a.N) *lane_of<float>(a.chunk, row + (int64_t)n * a.C, c4) = h[n];
  a.span[(int64_t)tile * a.C + c] = span;
  if (cb == 0 && lane == 0) {
    unsigned long long any = 0;
    const int at = t0 & 63;
    if (a.L < 64) any = G.first[0] >> at & ((1ull << a.L) - 1);
    else
      for (int k = 0; k < a.L / 64; ++k) any |= G.first[k];
    a.flag[tile] = any != 0;
  }
}

// The state before each tile (step 1), or the gradient of the state behind it
// (step -1), in place of the tile's own; one thread per channel and state.
__global__ void __launch_bounds__(kThreads) scan_chain_kernel(ScanArgs a, float *own,
                                                              const float *span,
                                                              const int32_t *flag, int step) {
  constexpr int U = 8;
  const int64_t n = (int64_t)a.N * a.C, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= n) return;
  const int c = (int)(id % a.C);
  const float A2 = a.a2[id];
  float carry = 0.f, o[U], s[U];
  int f[U];
  int64_t tile = step > 0 ? 0 : a.ntiles - 1;
  auto fetch = [&](int64_t from) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = from + u * step;
      const bool in = t >= 0 && t < a.ntiles;
      o[u] = in ? own[t * n + id] : 0.f;
      s[u] = in ? span[t * a.C + c] : 0.f;
      f[u] = in ? flag[t] : 0;
    }
  };
  for (int done = 0; done < a.ntiles; done += U, tile += U * step) {
    fetch(tile);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (done + u >= a.ntiles) break;
      own[(tile + u * step) * n + id] = carry;
      const float p = fmaxf(__builtin_amdgcn_exp2f(A2 * s[u]), kTiny);
      carry = f[u] ? o[u] : carry == 0.f ? o[u] : fmaf(p, carry, o[u]);
    }
  }
}

// --------------------------------------------------------------------- decode

// Q lanes per channel with four states each (N = 4 Q), U such quarters a thread, a
// workgroup apart: the state row is read, updated and written once, 16 bytes a
// lane for fp32 states, and the output is summed over the lanes.  Bounded by
// memory for a full batch (256 sequences of 4096 channels: 41 us, 28 at the rate of a
// large copy).
template <typename Tx, int Q, int U>
__global__ void __launch_bounds__(kThreads) scan_decode_kernel(ScanArgs a, int blocks) {
  if (blockIdx.x == 0 && a.b.status) decode_status(a.b);
  if (a.b.N == 0) return;
  const int i = blockIdx.x / blocks;
  const int per = a.C * Q, first = (int)(blockIdx.x % blocks) * (U * kThreads) + threadIdx.x;
  const int64_t r = state_row(a.b, i);
  float h[U][4], Av[U][4], Bv[U][4], Cv[U][4], x[U], d[U], z[U], D[U];
  int64_t on_a[U], on_b[U], on_h[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int at = min(first + k * kThreads, per - 1), c = at / Q, q = at % Q;
    on_a[k] = 4 * at;
    on_b[k] = (int64_t)(c / a.P) * a.N + 4 * q;
    on_h[k] = r * a.init.stride + 4 * at;
#pragma unroll
    for (int n = 0; n < 4; ++n) h[k][n] = 0.f;
    x[k] = to_f32(((const Tx *)a.x)[i * a.x_stride + c]);
    d[k] = to_f32(((const Tx *)a.delta)[i * a.delta_stride + c]) + (a.dbias ? a.dbias[c] : 0.f);
    z[k] = a.z ? to_f32(((const Tx *)a.z)[i * a.z_stride + c]) : 0.f;
    D[k] = a.D ? a.D[c] : 0.f;
  }
  rows_load<float, U, 4>(a.A, a.vec, on_a, Av);
  rows_load<Tx, U, 4>((const Tx *)a.B + i * a.b_stride, a.vec, on_b, Bv);
  rows_load<Tx, U, 4>((const Tx *)a.C_ + i * a.c_stride, a.vec, on_b, Cv);
  if (a.init.p && r >= 0) state_read<U, 4>(a.init, on_h, h);
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int at = first + k * kThreads;
    const bool on = at < per;
    const float dt = step_size(a, d[k]), u = dt * x[k];
    float y = 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      h[k][n] = fmaf(__builtin_amdgcn_exp2f(dt * (kLog2E * Av[k][n])), h[k][n], u * Bv[k][n]);
      y = fmaf(Cv[k][n], h[k][n], y);
    }
    if (a.fin.p && r >= 0 && on) {
      const int64_t to[1] = {r * a.fin.stride + 4 * at};
      const float(&row)[1][4] = reinterpret_cast<const float(&)[1][4]>(h[k]);
      state_write<1, 4>(a.fin, to, row);
    }
#pragma unroll
    for (int o = 1; o < Q; o <<= 1) y += __shfl_xor(y, o);
    if (!on || at % Q != 0) continue;
    if (a.D) y = fmaf(D[k], x[k], y);
    if (a.z) y *= z[k] * sigmoid(z[k]);
    ((Tx *)a.out)[(int64_t)i * a.C + at / Q] = from_f32<Tx>(y);
  }
}

// Any N: one lane per channel, one state after the other, each load behind the store
// before it (256 sequences of 4096 channels, states that a cache holds: 76 us with 12
// states and 652 with 33, where 16 take 25).
template <typename Tx>
__global__ void __launch_bounds__(kThreads) scan_decode_any_kernel(ScanArgs a, int blocks) {
  if (blockIdx.x == 0 && a.b.status) decode_status(a.b);
  if (a.b.N == 0) return;
  const int i = blockIdx.x / blocks, c = (int)(blockIdx.x % blocks) * kThreads + threadIdx.x;
  if (c >= a.C) return;
  const int64_t r = state_row(a.b, i), off = (int64_t)c * a.N, bn = (int64_t)(c / a.P) * a.N;
  const float x = to_f32(((const Tx *)a.x)[i * a.x_stride + c]);
  const float dt = step_size(a, to_f32(((const Tx *)a.delta)[i * a.delta_stride + c]) +
                                    (a.dbias ? a.dbias[c] : 0.f));
  const float u = dt * x;
  const Tx *B = (const Tx *)a.B + i * a.b_stride + bn, *C = (const Tx *)a.C_ + i * a.c_stride + bn;
  float y = 0.f;
  for (int n = 0; n < a.N; ++n) {
    float h[1][1] = {{0.f}};
    const int64_t from[1] = {r * a.init.stride + off + n}, to[1] = {r * a.fin.stride + off + n};
    if (a.init.p && r >= 0) state_read<1, 1>(a.init, from, h);
    h[0][0] = fmaf(__builtin_amdgcn_exp2f(dt * (kLog2E * a.A[off + n])), h[0][0], u * to_f32(B[n]));
    y = fmaf(to_f32(C[n]), h[0][0], y);
    if (a.fin.p && r >= 0) state_write<1, 1>(a.fin, to, h);
  }
  if (a.D) y = fmaf(a.D[c], x, y);
  if (a.z) {
    const float z = to_f32(((const Tx *)a.z)[i * a.z_stride + c]);
    y *= z * sigmoid(z);
  }
  ((Tx *)a.out)[(int64_t)i * a.C + c] = from_f32<Tx>(y);
}

// ------------------------------------------------------------------- launches

template <typename Tx, int NS> struct States {
  static hipError_t go(const ScanArgs &a, hipStream_t s) {
    // (which leaves no more than N states, and no sums over them)
    scan_tile_kernel<Tx, NS, false, true><<<dim3(tile_grid(a, 0)), dim3(kThreads), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? launch_scan_chain(a, false, s) : e;
  }
};
template <typename Tx, int NS> struct Forward {
  static hipError_t go(const ScanArgs &a, hipStream_t s) {
    const dim3 grid(tile_grid(a, a.empties));
    if (a.N == NS) scan_tile_kernel<Tx, NS, true, true><<<grid, dim3(kThreads), 0, s>>>(a);
    else scan_tile_kernel<Tx, NS, true, false><<<grid, dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
  }
};
template <typename Tx> hipError_t prepare(const ScanArgs &a, hipStream_t s) {
  const int ns = scan_states(a.N);
  const int64_t n = std::max<int64_t>(a.b.T * a.G * 2 * ns, (int64_t)ns * a.C);
  const int64_t want = (n + 4 * kThreads - 1) / (4 * kThreads), most = 8 * (int64_t)a.num_cus;
  scan_prepare_kernel<Tx><<<dim3((unsigned)std::min(want, most)), dim3(kThreads), 0, s>>>(a, ns);
  return hipGetLastError();
}

template <typename Tx, int Q> hipError_t decode_by(const ScanArgs &a, hipStream_t s) {
  // four quarters a thread where that leaves two workgroups per CU
  constexpr int U = 4;
  const int64_t per = (int64_t)a.C * Q, n = std::max<int64_t>(a.b.N, 1);
  const int64_t long_ = (per + U * kThreads - 1) / (U * kThreads);
  if (long_ * n >= 2 * (int64_t)a.num_cus) {
    scan_decode_kernel<Tx, Q, U>
        <<<dim3((unsigned)(long_ * n)), dim3(kThreads), 0, s>>>(a, (int)long_);
  } else {
    const int64_t blocks = (per + kThreads - 1) / kThreads;
    scan_decode_kernel<Tx, Q, 1>
        <<<dim3((unsigned)(blocks * n)), dim3(kThreads), 0, s>>>(a, (int)blocks);
  }
  return hipGetLastError();
}
template <typename Tx> hipError_t decode(const ScanArgs &a, hipStream_t s) {
  switch (a.N) {
    case 4: return decode_by<Tx, 1>(a, s);
    case 8: return decode_by<Tx, 2>(a, s);
    case 16: return decode_by<Tx, 4>(a, s);
    case 32: return decode_by<Tx, 8>(a, s);
    case 64: return decode_by<Tx, 16>(a, s);
    default: break;
  }
  const int64_t blocks = (a.C + kThreads - 1) / kThreads, n = std::max<int64_t>(a.b.N, 1);
  scan_decode_any_kernel<Tx>
      <<<dim3((unsigned)(blocks * n)), dim3(kThreads), 0, s>>>(a, (int)blocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_prepare(const ScanArgs &a, hipStream_t s) {
  if (a.x_dtype == GDN_F32) return prepare<float>(a, s);
  return a.x_dtype == GDN_BF16 ? prepare<bf16>(a, s) : prepare<f16>(a, s);
}
hipError_t launch_scan_chain(const ScanArgs &a, bool backward, hipStream_t s) {
  const int64_t n = (int64_t)a.N * a.C;
  const dim3 grid((unsigned)((n + kThreads - 1) / kThreads));
  if (backward)
    scan_chain_kernel<<<grid, dim3(kThreads), 0, s>>>(a, a.gchunk, a.gspan, a.gflag, -1);
  else
    scan_chain_kernel<<<grid, dim3(kThreads), 0, s>>>(a, a.chunk, a.span, a.flag, 1);
  return hipGetLastError();
}
hipError_t launch_scan_states(const ScanArgs &a, hipStream_t s) { return dispatch<States>(a, s); }
hipError_t launch_scan_forward(const ScanArgs &a, hipStream_t s) { return dispatch<Forward>(a, s); }
hipError_t launch_scan_decode(const ScanArgs &a, hipStream_t s) {
  if (a.x_dtype == GDN_F32) return decode<float>(a, s);
  return a.x_dtype == GDN_BF16 ? decode<bf16>(a, s) : decode<f16>(a, s);
}

}  // namespace gdn
