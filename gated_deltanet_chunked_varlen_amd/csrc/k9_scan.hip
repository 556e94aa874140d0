// k9_scan.hip -- selective state space scan of packed sequences: forward,
// backward and decode step.
//
// With step size d_t = softplus(delta_t + delta_bias) (or as given), for every
// channel c and each of its N states n, in fp32,
//     h_t = exp(d_t A) h_{t-1} + d_t B_t x_t
//     y_t = sum_n C_t h_t + D x_t,     output_t = y_t silu(z_t)
//
// Bounded by the vector ALU: a token takes, for each state, the exponential (the
// cost of two other operations), its argument, the input's product and two
// fused products, 24 cycles of a SIMD per 64 states, against 8 bytes of a
// channel's token for all of its states.  So a lane holds one channel with all of
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
// initial states.
__device__ __forceinline__ void empty_sequences(const ScanArgs &a, int part) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)a.C * a.N;
  for (int i = part; i < a.b.N; i += a.empties) {
    int bos, len;
    sequence_of(a.b, i, lane, bos, len);
    if (len != 0) continue;
    const int64_t r = state_row(a.b, i);
    if (r < 0) continue;
    for (int64_t e = threadIdx.x; e < row; e += kThreads) {
      float one[1] = {0.f};
      if (a.init.p) state_read<1>(a.init, r * a.init.stride + e, one);
      state_write<1>(a.fin, r * a.fin.stride + e, one);
    }
  }
}

// OUT false: a tile's own last state, the sum of its step sizes, and the initial
// state of a sequence that starts in it and goes on.  OUT true: outputs and
// final states from the state before the tile.
template <typename Tx, int NS, bool OUT>
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
    if (OUT && blockIdx.x % ncw == 0 && tile - a.ntiles < a.empties)
      empty_sequences(a, tile - a.ntiles);
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
    auto token = [&](int u, float x, float dt, float z) {
      float y = D * x;
      token_step<NS, OUT>(bc + (t + u) * bcs, dt, dt * x, A2, h, y);
      if (OUT) {
        if (a.z) y *= z * sigmoid(z);
        if (ch.ok) *lane_of<Tx>(a.out, (int64_t)(t + u) * a.C, (unsigned)c * sizeof(Tx)) = from_f32<Tx>(y);
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
#pragma unroll 4
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
#pragma unroll 4
          for (int n = 0; n < a.N; ++n)
            *lane_of<float>(a.start, row + (int64_t)n * a.C, c4) = lds[n * 64];
        }
        span = 0.f;
      }
      token(u, run[u * 64], run[(kRun + u) * 64], OUT ? run[(2 * kRun + u) * 64] : 0.f);
      if (OUT && a.fin.p && ch.ok && (m.last >> u & 1)) final_state<NS>(a, m.seq_at(u), c, lds, h);
    }
  }
  if (OUT || !ch.ok) return;
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

// Q lanes per channel with four states each (N = 4 Q): the state row is read,
// updated and written once, 16 bytes a lane for fp32 states, and the output is
// summed over the lanes.  Bounded by memory for a full batch.  Q = 0: one lane
// per channel, any N.
template <typename Tx, int Q>
__global__ void __launch_bounds__(kThreads) scan_decode_kernel(ScanArgs a) {
  constexpr int S = Q ? Q : 1;
  if (blockIdx.x == 0 && a.b.status) decode_status(a.b);
  const int64_t per = (int64_t)a.C * S;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const bool on = id < per * a.b.N;
  const int i = on ? (int)(id / per) : 0;
  const int64_t at = on ? id % per : 0;
  const int c = (int)(at / S), q = (int)(at % S);
  const int64_t r = on ? state_row(a.b, i) : -1;
  float x = 0.f, dt = 0.f, y = 0.f;
  if (on) {
    x = to_f32(((const Tx *)a.x)[i * a.x_stride + c]);
    dt = step_size(a, to_f32(((const Tx *)a.delta)[i * a.delta_stride + c]) +
                          (a.dbias ? a.dbias[c] : 0.f));
    const float u = dt * x;
    const int64_t bn = (int64_t)(c / a.P) * a.N;
    const Tx *B = (const Tx *)a.B + i * a.b_stride + bn, *C = (const Tx *)a.C_ + i * a.c_stride + bn;
    const float *A = a.A + (int64_t)c * a.N;
    const int64_t off = (int64_t)c * a.N;
    if constexpr (Q > 0) {
      float h[4] = {0.f, 0.f, 0.f, 0.f}, Av[4], Bv[4], Cv[4];
      if (a.init.p && r >= 0) state_read<4>(a.init, r * a.init.stride + off + 4 * q, h);
      row_load<float, 4>(A, 4 * q, Av);
      row_load<Tx, 4>(B, 4 * q, Bv);
      row_load<Tx, 4>(C, 4 * q, Cv);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        h[n] = fmaf(__builtin_amdgcn_exp2f(dt * (kLog2E * Av[n])), h[n], u * Bv[n]);
        y = fmaf(Cv[n], h[n], y);
      }
      if (a.fin.p && r >= 0) state_write<4>(a.fin, r * a.fin.stride + off + 4 * q, h);
    } else {
      for (int n = 0; n < a.N; ++n) {
        float h[1] = {0.f};
        if (a.init.p && r >= 0) state_read<1>(a.init, r * a.init.stride + off + n, h);
        h[0] = fmaf(__builtin_amdgcn_exp2f(dt * (kLog2E * A[n])), h[0], u * to_f32(B[n]));
        y = fmaf(to_f32(C[n]), h[0], y);
        if (a.fin.p && r >= 0) state_write<1>(a.fin, r * a.fin.stride + off + n, h);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < S; o <<= 1) y += __shfl_xor(y, o);
  if (!on || q != 0) return;
  y = fmaf(a.D ? a.D[c] : 0.f, x, y);
  if (a.z) {
    const float z = to_f32(((const Tx *)a.z)[i * a.z_stride + c]);
    y *= z * sigmoid(z);
  }
  ((Tx *)a.out)[(int64_t)i * a.C + c] = from_f32<Tx>(y);
}

// ------------------------------------------------------------------- launches

template <typename Tx, int NS> struct States {
  static hipError_t go(const ScanArgs &a, hipStream_t s) {
    scan_tile_kernel<Tx, NS, false><<<dim3(tile_grid(a, 0)), dim3(kThreads), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? launch_scan_chain(a, false, s) : e;
  }
};
template <typename Tx, int NS> struct Forward {
  static hipError_t go(const ScanArgs &a, hipStream_t s) {
    scan_tile_kernel<Tx, NS, true><<<dim3(tile_grid(a, a.empties)), dim3(kThreads), 0, s>>>(a);
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

template <typename Tx> hipError_t decode(const ScanArgs &a, hipStream_t s) {
  const int q = a.N == 4 ? 1 : a.N == 8 ? 2 : a.N == 16 ? 4 : a.N == 32 ? 8 : a.N == 64 ? 16 : 0;
  const int64_t n = (int64_t)a.b.N * a.C * (q ? q : 1);
  const dim3 grid((unsigned)(n > 0 ? (n + kThreads - 1) / kThreads : 1)), block(kThreads);
  if (q == 1) scan_decode_kernel<Tx, 1><<<grid, block, 0, s>>>(a);
  else if (q == 2) scan_decode_kernel<Tx, 2><<<grid, block, 0, s>>>(a);
  else if (q == 4) scan_decode_kernel<Tx, 4><<<grid, block, 0, s>>>(a);
  else if (q == 8) scan_decode_kernel<Tx, 8><<<grid, block, 0, s>>>(a);
  else if (q == 16) scan_decode_kernel<Tx, 16><<<grid, block, 0, s>>>(a);
  else scan_decode_kernel<Tx, 0><<<grid, block, 0, s>>>(a);
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
