// k10_scan_backward.hip -- backward pass of the selective state space scan.
//
// With y' the gradient of y (doutput silu(z)) and g the gradient of a state:
//     g_t = C_t y'_t + exp(d_{t+1} A) g_{t+1}     (last token: + dfinal)
//     dC_t = sum_c y'_t h_t,   dB_t = sum_c g_t d_t x_t
//     du_t = sum_n g_t B_t,    r_t = g_t exp(d_t A) h_{t-1}
//     dx_t = du_t d_t + D y'_t,   dd_t = du_t x_t + sum_n r_t A
//     dA = sum_t r_t d_t,   dD = sum_t y'_t x_t
// The kernels: every tile's own gradient of the state before it, the chain from
// the last tile to the first, then the tiles.  A tile forms its states again
// from the one before it, in blocks of kBlock tokens: first the states before
// each block (into LDS), then, from the last block to the first and one state n
// after the other, the block's states and gradients in registers.  Sums over
// the channels of a block of 64 are formed by lane moves that keep half of the
// values at each step, stored, and added by a last kernel, in a fixed order.
//
// Bounded by the vector ALU (half of the time) and by the waits of two waves per
// SIMD: 4096 tokens of 4096 channels with 16 states in bf16 take 457 us, in parts
// that overlap some 290 the loop over the states, 155 raw values and results, 45 the
// states before the blocks; the gradients before the tiles 71 and the chain 14.  With
// the gradients behind a block in LDS of their own, one workgroup less per CU, it was
// 700.  With 64 states a tile has 16 tokens, so that the states and sums of tiles are
// most of the traffic, and a few registers are spilled: the whole pass takes 1.93 ms
// there, 0.50 with 16 states.

#include "gdn_scan.h"

#include <atomic>
#include <type_traits>

#pragma clang fp contract(off)

namespace gdn {

using namespace scan;

namespace {

constexpr int kBlock = 16;
constexpr int kPart = 8;  // tokens whose raw values are held at once

// Gradients of the empty sequences' initial states: those of their final states.
// A row of workgroups (`slice` of `slices`) takes every a.empties-th sequence.
__device__ __forceinline__ void empty_sequences(const ScanArgs &a, int part, int slice,
                                                int slices) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)a.C * a.N, step = (int64_t)slices * kThreads;
  for (int i = part; i < a.b.N; i += a.empties) {
    int bos, len;
    sequence_of(a.b, i, lane, bos, len);
    if (len != 0) continue;
#pragma unroll 4
    for (int64_t e = slice * kThreads + threadIdx.x; e < row; e += step)
      a.dinit[i * row + e] = a.dfin ? a.dfin[i * row + e] : 0.f;
  }
}

// State n of sequence i, channel c, before its first token.
__device__ __forceinline__ float initial_state(const ScanArgs &a, int i, int c, int n) {
  return a.init.p ? ((const float *)a.init.p)[i * a.init.stride + (int64_t)c * a.N + n] : 0.f;
}

// y' of a token.
__device__ __forceinline__ float output_gradient(const ScanArgs &a, float dy, float z) {
  return a.z ? dy * (z * sigmoid(z)) : dy;
}

template <typename Tx, int NS>
__global__ void __launch_bounds__(kThreads, scan_waves(NS)) scan_gradient_kernel(ScanArgs a) {
  __shared__ TileGeo G;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ncw = (a.ncb + kWaves - 1) / kWaves;
  const int tile = blockIdx.x / ncw, t0 = tile * a.L;
  tile_geometry(a, t0, G);
  const int cb = (int)(blockIdx.x % ncw) * kWaves + wave;
  if (cb >= a.ncb) return;
  const Channel ch(a, cb, lane);
  const unsigned c4 = (unsigned)ch.c * 4;
  const int c = ch.c, end = (int)a.b.T - 1;
  constexpr int Q = NS < 16 ? NS : 16;
  typedef float vec __attribute__((ext_vector_type(Q)));
  float A2[NS], g[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    A2[n] = *lane_of<float>(a.a2, (int64_t)n * a.C, c4);
    g[n] = 0.f;
  }
  const float bias = a.dbias ? a.dbias[c] : 0.f;
  const float *cs = a.bc + (int64_t)ch.g * 2 * NS + NS;
  const int64_t bcs = (int64_t)a.G * 2 * NS;
  float span = 0.f;
  const int L = min(a.L, (int)a.b.T - t0);
  for (int s = (L - 1) / kRun * kRun; s >= 0; s -= kRun) {
    const int t = t0 + s;
    const Marks m(G, (t0 & 63) + s, kRun);
    Rows<Tx, kRun> ry, rd, rz;
    ry.load(a.dy, a.dy_stride, t, end, c);
    rd.load(a.delta, a.delta_stride, t, end, c);
    if (a.z) rz.load(a.z, a.z_stride, t, end, c);
    float y[kRun], dt[kRun];
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      y[u] = output_gradient(a, to_f32(ry.v[u]), a.z ? to_f32(rz.v[u]) : 0.f);
      dt[u] = step_size(a, to_f32(rd.v[u]) + bias);
    }
    auto token = [&](int u) {
#pragma unroll
      for (int k = 0; k < NS; k += Q) {
        const vec cc = uniform_load<vec>(cs + (t + u) * bcs + k);
#pragma unroll
        for (int n = 0; n < Q; ++n)
          g[k + n] = __builtin_amdgcn_exp2f(dt[u] * A2[k + n]) * fmaf(cc[n], y[u], g[k + n]);
      }
      span += dt[u];
    };
    if (m.valid == (1u << kRun) - 1 && m.last == 0) {
#pragma unroll
      for (int u = kRun - 1; u >= 0; --u) token(u);
      continue;
    }
#pragma unroll 1
    for (int u = kRun - 1; u >= 0; --u) {
      if (!(m.valid >> u & 1)) continue;
      if (m.last >> u & 1) {
        const int64_t off = ((int64_t)m.seq_at(u) * a.C + c) * a.N;
#pragma unroll
        for (int n = 0; n < NS; ++n) g[n] = a.dfin && n < a.N ? a.dfin[off + n] : 0.f;
        span = 0.f;
      }
      token(u);
    }
  }
  if (!ch.ok) return;
  const int64_t row = (int64_t)tile * a.N * a.C;
#pragma unroll
  for (int n = 0; n < NS; ++n)
    if (n < a.N) *lane_of<float>(a.gchunk, row + (int64_t)n * a.C, c4) = g[n];
  a.gspan[(int64_t)tile * a.C + c] = span;
  if (cb == 0 && lane == 0) {
    unsigned long long any = 0;
    const int at = t0 & 63;
    if (a.L < 64) any = G.last[0] >> at & ((1ull << a.L) - 1);
    else
      for (int k = 0; k < a.L / 64; ++k) any |= G.last[k];
    a.gflag[tile] = any != 0;
  }
}

template <int CTRL> __device__ __forceinline__ float moved(float x) {
  return __uint_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xF, 0xF, true));
}

// Sums of 32 values over the wave's lanes: lane l receives the sum of value l / 2.
// Each step adds the lanes of a pair and keeps one value for each of them: half
// as many registers after it.
__device__ __forceinline__ float sums_of_32(float (&v)[32], int lane) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]),
                                                    __float_as_uint(v[i + 16]), false, false);
    v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]),
                                                    __float_as_uint(v[i + 8]), false, false);
    v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  const bool b3 = lane & 8, b2 = lane & 4, b1 = lane & 2;
#pragma unroll
  for (int i = 0; i < 4; ++i)  // lane xor 8
    v[i] = (b3 ? v[i + 4] : v[i]) + moved<0x128>(b3 ? v[i] : v[i + 4]);
#pragma unroll
  for (int i = 0; i < 2; ++i)  // lane xor 7
    v[i] = (b2 ? v[i + 2] : v[i]) + moved<0x141>(b2 ? v[i] : v[i + 2]);
  // lane xor 2, lane xor 1
  const float s = (b1 ? v[1] : v[0]) + moved<0x4E>(b1 ? v[0] : v[1]);
  return s + moved<0xB1>(s);
}

template <typename Tx, int NS>
__global__ void __launch_bounds__(kThreads, 2) scan_backward_kernel(ScanArgs a) {
  __shared__ TileGeo G;
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ncw = (a.ncb + kWaves - 1) / kWaves;
  const int tile = blockIdx.x / ncw, t0 = tile * a.L;
  if (blockIdx.x == 0 && wave == 0 && a.b.status && !a.b.bos) batch_status(a.b, lane);
  if (tile >= a.ntiles) {
    if (tile - a.ntiles < a.empties)
      empty_sequences(a, tile - a.ntiles, blockIdx.x % ncw, ncw);
    return;
  }
  tile_geometry(a, t0, G);
  const int cb = (int)(blockIdx.x % ncw) * kWaves + wave;
  if (cb >= a.ncb) return;
  const Channel ch(a, cb, lane);
  const unsigned c4 = (unsigned)ch.c * 4;
  const int c = ch.c, end = (int)a.b.T - 1, blocks = a.L / kBlock;
  // this wave's LDS: the states before blocks 1 .. (once used, the gradients behind
  // the block before), and dA of each state
  float *const st = lds + (int64_t)wave * blocks * NS * 64 + lane;
  float *const as = st + (int64_t)(blocks - 1) * NS * 64;
  const float bias = a.dbias ? a.dbias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
  const int64_t row = (int64_t)tile * a.N * a.C;
  const bool chained = a.ntiles > 1;
  const int used = (min(a.L, (int)a.b.T - t0) + kBlock - 1) / kBlock;  // blocks with tokens

  {  // the states before the blocks
    float A2[NS], h[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      A2[n] = *lane_of<float>(a.a2, (int64_t)n * a.C, c4);
      h[n] = chained && n < a.N ? *lane_of<float>(a.chunk, row + (int64_t)n * a.C, c4) : 0.f;
    }
    const float *bc = a.bc + (int64_t)ch.g * 2 * NS;
    const int64_t bcs = (int64_t)a.G * 2 * NS;
    for (int s = 0; s < (used - 1) * kBlock; s += kRun) {
      const int t = t0 + s;
      const Marks m(G, (t0 & 63) + s, kRun);
      Rows<Tx, kRun> rx, rd;
      rx.load(a.x, a.x_stride, t, end, c);
      rd.load(a.delta, a.delta_stride, t, end, c);
      float none = 0.f, x[kRun], dt[kRun];
#pragma unroll
      for (int u = 0; u < kRun; ++u) {
        x[u] = to_f32(rx.v[u]);
        dt[u] = step_size(a, to_f32(rd.v[u]) + bias);
      }
      auto token = [&](int u) {
        token_step<NS, false>(bc + (t + u) * bcs, dt[u], dt[u] * x[u], A2, h, none);
      };
      if (m.valid == (1u << kRun) - 1 && m.first == 0) {
#pragma unroll
        for (int u = 0; u < kRun; ++u) token(u);
      } else {
#pragma unroll 1
        for (int u = 0; u < kRun; ++u) {
          if (!(m.valid >> u & 1)) continue;
          if (m.first >> u & 1) {
            const int i = m.seq_at(u);
#pragma unroll
            for (int n = 0; n < NS; ++n) h[n] = n < a.N ? initial_state(a, i, c, n) : 0.f;
          }
          token(u);
        }
      }
      if ((s + kRun) % kBlock == 0) {
        float *o = st + (int64_t)((s + kRun) / kBlock - 1) * NS * 64;
#pragma unroll
        for (int n = 0; n < NS; ++n) o[n * 64] = h[n];
      }
    }
  }
  // the gradients behind the tile wait in dA's place, which is not used before them
  if (chained) {
#pragma unroll
    for (int n = 0; n < NS; ++n)
      if (n < a.N) as[n * 64] = *lane_of<float>(a.gchunk, row + (int64_t)n * a.C, c4);
  } else {
#pragma unroll
    for (int n = 0; n < NS; ++n) as[n * 64] = 0.f;
  }
  float dD = 0.f, dbias = 0.f;
  for (int blk = used - 1; blk >= 0; --blk) {
    const int tb = t0 + blk * kBlock;
    const Marks m(G, (t0 & 63) + blk * kBlock, kBlock);
    const bool newest = blk == used - 1;
    float dt[kBlock], u[kBlock], y[kBlock], du[kBlock], dd[kBlock], yy[kBlock];
#pragma unroll
    for (int k = 0; k < kBlock; k += kPart) {
      Rows<Tx, kPart> rx, rd, ry, rz;
      rx.load(a.x, a.x_stride, tb + k, end, c);
      rd.load(a.delta, a.delta_stride, tb + k, end, c);
      ry.load(a.dy, a.dy_stride, tb + k, end, c);
      if (a.z) rz.load(a.z, a.z_stride, tb + k, end, c);
#pragma unroll
      for (int j = 0; j < kPart; ++j) {
        const int i = k + j;
        const bool in = ch.ok && (m.valid >> i & 1);
        dt[i] = in ? step_size(a, to_f32(rd.v[j]) + bias) : 0.f;
        u[i] = in ? dt[i] * to_f32(rx.v[j]) : 0.f;
        y[i] = in ? output_gradient(a, to_f32(ry.v[j]), a.z ? to_f32(rz.v[j]) : 0.f) : 0.f;
        du[i] = dd[i] = yy[i] = 0.f;
      }
    }
    auto states = [&](auto plain) {
      constexpr bool PLAIN = decltype(plain)::value;
      // what state n starts from, read while the state before it is worked on
      struct Start {
        float A2, h, g;
        f32x16 bb;
      };
      const int64_t at0 = (int64_t)ch.g * 2 * NS * a.Tp + tb;
      auto start_of = [&](int n) {
        Start o;
        o.A2 = *lane_of<float>(a.a2, (int64_t)n * a.C, c4);
        o.bb = uniform_load<f32x16>(a.bct + at0 + (int64_t)n * a.Tp);
        o.h = blk > 0  ? st[((blk - 1) * NS + n) * 64]
              : chained ? *lane_of<float>(a.chunk, row + (int64_t)n * a.C, c4)
                        : 0.f;
        o.g = newest ? as[n * 64] : st[(blk * NS + n) * 64];
        return o;
      };
      Start now = start_of(0);
#pragma unroll 1
      for (int n = 0; n < a.N; ++n) {
        const float A2 = now.A2;
        const f32x16 cc = uniform_load<f32x16>(a.bct + at0 + (int64_t)(NS + n) * a.Tp);
        float h = now.h, g = now.g;
        float e[kBlock], before[kBlock + 1], v[2 * kBlock];
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
          v[i] = v[kBlock + i] = 0.f;
          if (!PLAIN) {
            e[i] = before[i] = 0.f;
            if (!(m.valid >> i & 1)) continue;
            if (m.first >> i & 1) h = initial_state(a, m.seq_at(i), c, n);
          }
          before[i] = h;
          e[i] = __builtin_amdgcn_exp2f(dt[i] * A2);
          h = fmaf(e[i], h, u[i] * now.bb[i]);
          v[kBlock + i] = y[i] * h;
          if (!PLAIN) yy[i] = fmaf(cc[i], h, yy[i]);
        }
        before[kBlock] = h;
        const Start next = start_of(min(n + 1, a.N - 1));
        float dA = 0.f;
#pragma unroll
        for (int i = kBlock - 1; i >= 0; --i) {
          if (!PLAIN) {
            if (!(m.valid >> i & 1)) continue;
            if (m.last >> i & 1)
              g = a.dfin ? a.dfin[((int64_t)m.seq_at(i) * a.C + c) * a.N + n] : 0.f;
          }
          if (PLAIN) yy[i] = fmaf(cc[i], before[i + 1], yy[i]);
          g = fmaf(cc[i], y[i], g);
          v[i] = g * u[i];
          du[i] = fmaf(g, now.bb[i], du[i]);
          g *= e[i];
          const float r = g * before[i];
          dd[i] = fmaf(r, A2, dd[i]);
          dA = fmaf(r, dt[i], dA);
          if (!PLAIN && a.dinit && ch.ok && (m.first >> i & 1))
            a.dinit[((int64_t)m.seq_at(i) * a.C + c) * a.N + n] = g;
        }
        if (blk > 0) st[((blk - 1) * NS + n) * 64] = g;
        as[n * 64] = newest ? dA : as[n * 64] + dA;
        now = next;
        if (!ch.ok) {
#pragma unroll
          for (int i = 0; i < 2 * kBlock; ++i) v[i] = 0.f;
        }
        const float sum = sums_of_32(v, lane);
        const int k = lane >> 1;  // dB of tokens 0 .. 15, then dC
        if ((lane & 1) == 0)
          a.pbc[(((int64_t)cb * 2 + (k >> 4)) * NS + n) * a.Tp + tb + (k & 15)] = sum;
      }
    };
    if (m.valid == (1u << kBlock) - 1 && (m.first | m.last) == 0) states(std::true_type{});
    else states(std::false_type{});
    // the inputs again: the compiler is not to know that it has seen them, or it
    // keeps all of them in registers (and others in memory)
    const void *xs = a.x, *ds = a.delta, *ys = a.dy, *zs = a.z;
    asm volatile("" : "+s"(xs), "+s"(ds), "+s"(ys), "+s"(zs));
    const int64_t first_row = (int64_t)tb * a.C * (int)sizeof(Tx);
    char *const orow[3] = {uniform((char *)a.dx + first_row), uniform((char *)a.ddelta + first_row),
                           uniform((char *)a.dz + first_row)};
    const unsigned cx = (unsigned)c * (unsigned)sizeof(Tx);
#pragma unroll
    for (int k = 0; k < kBlock; k += kPart) {
      Rows<Tx, kPart> rx, rd, ry, rz;
      rx.load(xs, a.x_stride, tb + k, end, c);
      if (a.softplus) rd.load(ds, a.delta_stride, tb + k, end, c);
      if (a.z) {
        ry.load(ys, a.dy_stride, tb + k, end, c);
        rz.load(zs, a.z_stride, tb + k, end, c);
      }
#pragma unroll
      for (int j = 0; j < kPart; ++j) {
        const int i = k + j;
        if (tb + i > end || !ch.ok) continue;
        const bool in = m.valid >> i & 1;
        const int64_t at = (int64_t)i * a.C * (int)sizeof(Tx);
        const float x = to_f32(rx.v[j]);
        float ddt = fmaf(du[i], x, kLn2 * dd[i]);
        if (a.softplus) ddt *= sigmoid(to_f32(rd.v[j]) + bias);
        const float dx = fmaf(du[i], dt[i], skip_of(a, D, y[i]));
        *(Tx *)(orow[0] + at + cx) = from_f32<Tx>(in ? dx : 0.f);
        *(Tx *)(orow[1] + at + cx) = from_f32<Tx>(in ? ddt : 0.f);
        if (a.z) {
          const float z = to_f32(rz.v[j]), sg = sigmoid(z);
          const float out = a.D ? fmaf(D, x, yy[i]) : yy[i];
          const float dz = to_f32(ry.v[j]) * out * (sg * fmaf(z, 1.f - sg, 1.f));
          *(Tx *)(orow[2] + at + cx) = from_f32<Tx>(in ? dz : 0.f);
        }
        if (in) {
          dD = fmaf(y[i], x, dD);
          dbias += ddt;
        }
      }
    }
  }
  if (!ch.ok) return;
  float *ps = a.psum + (int64_t)tile * (a.N + 2) * a.C + c;
  for (int n = 0; n < a.N; ++n) ps[(int64_t)n * a.C] = as[n * 64];
  ps[(int64_t)a.N * a.C] = dD;
  ps[(int64_t)(a.N + 1) * a.C] = dbias;
}

// dA, dD and ddelta_bias: the tiles' sums, added in order by eight threads a
// column (and then over these).
__global__ void __launch_bounds__(kThreads) scan_sums_kernel(ScanArgs a) {
  constexpr int kCols = 32, kParts = kThreads / kCols;
  __shared__ float sums[kParts][kCols];
  const int col = threadIdx.x % kCols, part = threadIdx.x / kCols;
  const int64_t n = (int64_t)(a.N + 2) * a.C, id = (int64_t)blockIdx.x * kCols + col;
  float sum = 0.f;
  if (id < n) {
#pragma unroll 4
    for (int r = part; r < a.ntiles; r += kParts) sum += a.psum[r * n + id];
  }
  sums[part][col] = sum;
  __syncthreads();
  if (part != 0 || id >= n) return;
#pragma unroll
  for (int p = 1; p < kParts; ++p) sum += sums[p][col];
  const int k = (int)(id / a.C), c = (int)(id % a.C);
  if (k < a.N) a.dA[(int64_t)c * a.N + k] = sum;
  else if (k == a.N) {
    if (a.dD) a.dD[c] = sum;
  } else if (a.ddbias) {
    a.ddbias[c] = sum;
  }
}

// dB and dC: the blocks of 64 channels of a group added in order.
template <typename Tx>
__global__ void __launch_bounds__(kThreads) scan_bc_sums_kernel(ScanArgs a, int ns) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t t = id % a.Tp;
  const int64_t row = id / a.Tp;  // (g, which, n), n < N
  if (row >= (int64_t)a.G * 2 * a.N || t >= a.b.T) return;
  const int n = (int)(row % a.N), which = (int)(row / a.N) % 2, g = (int)(row / (2 * a.N));
  const int per = a.ncb / a.G;
  float sum = 0.f;
#pragma unroll 4
  for (int k = 0; k < per; ++k)
    sum += a.pbc[(((int64_t)(g * per + k) * 2 + which) * ns + n) * a.Tp + t];
  ((Tx *)(which ? a.dC : a.dB))[(t * a.G + g) * a.N + n] = from_f32<Tx>(sum);
}

template <typename Tx, int NS> struct Backward {
  static hipError_t go(const ScanArgs &a, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (a.ntiles > 1) {
      scan_gradient_kernel<Tx, NS><<<dim3(tile_grid(a, 0)), dim3(kThreads), 0, s>>>(a);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      e = launch_scan_chain(a, true, s);
      if (e != hipSuccess) return e;
    }
    static std::atomic<uint64_t> done{0};
    const int lds = kWaves * (a.L / kBlock) * NS * 64 * (int)sizeof(float);
    e = set_dynamic_lds((const void *)scan_backward_kernel<Tx, NS>, 96 << 10, done);
    if (e != hipSuccess) return e;
    scan_backward_kernel<Tx, NS><<<dim3(tile_grid(a, a.empties)), dim3(kThreads), lds, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t cols = (int64_t)(a.N + 2) * a.C;
    scan_sums_kernel<<<dim3((unsigned)((cols + 31) / 32)), dim3(kThreads), 0, s>>>(a);
    e = hipGetLastError();
    const int64_t m = (int64_t)a.G * 2 * a.N * a.Tp;
    if (e != hipSuccess || m == 0) return e;
    scan_bc_sums_kernel<Tx>
        <<<dim3((unsigned)((m + kThreads - 1) / kThreads)), dim3(kThreads), 0, s>>>(a, NS);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_scan_backward(const ScanArgs &a, hipStream_t s) {
  return dispatch<Backward>(a, s);
}

}  // namespace gdn
