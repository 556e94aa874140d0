// gdn_layers.h -- argument blocks, launchers and device-side building blocks of
// the operators around a recurrence: the short causal convolution, the
// selective state space scan and beam search over state pools.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gdn_prefill.h"
#include "gdn_common.h"
#include "gdn_internal.h"

namespace gdn {

// A packed batch: sequence bounds and state rows.
struct Batch {
  int64_t T;
  int32_t N;
  const void *cu;  // cu_seqlens; NULL: one sequence [0, T]
  int32_t cu_type;
  const int32_t *bos;  // sanitised sequence starts [N + 1]; NULL: N <= 63, from cu
  const void *sidx;    // state rows; NULL: row i
  int32_t sidx_type;
  int64_t pool_rows;
  int32_t *status;
};

// Rows of states of any state dtype, `stride` elements apart.  vec: rows, and the
// rows of channels that one is made of, are whole aligned groups of 16 bytes.
struct StateRows {
  void *p;
  int32_t dtype, vec;
  int64_t stride;
};

// Channels that a lane of the convolution's kernels takes at a time (mode: forward,
// backward, decode), of es bytes each: 16 bytes, but in the backward pass, which
// holds three rows of sums for each of them, four (packed batch of 23 060 x 8192 in
// bf16: 307 us, 342 with eight).
constexpr int conv_lane(int mode, int es) { return mode == 1 ? 4 : 16 / es; }

struct ConvArgs {
  Batch b;
  int32_t C, W;
  int32_t x_dtype, w_dtype, silu;
  const void *x;
  int64_t x_stride;
  const void *w, *bias;
  void *out;
  StateRows init, fin;
  // backward
  const void *dy;
  int64_t dy_stride;
  const float *dfin;
  void *dx;
  float *dw, *db, *dinit;
  float *part;  // [runs][W + 1][C] sums of one run of tokens
  // cut: runs of `run` tokens by blocks of 64 lanes x vec channels
  int32_t run, runs, ncb, vec;
  int32_t fvec;  // fp32 rows of channels (dfin, dinit, part) are aligned groups of 16 bytes
};

hipError_t launch_conv_forward(const ConvArgs &a, hipStream_t s);
hipError_t launch_conv_backward(const ConvArgs &a, hipStream_t s);
hipError_t launch_conv_decode(const ConvArgs &a, hipStream_t s);

struct ScanArgs {
  Batch b;
  int32_t C, N, G;     // channels, states of a channel, groups of channels
  int32_t P, ncb;      // channels of a group, blocks of 64 channels (per group whole ones)
  int32_t x_dtype, softplus;
  const void *x, *delta, *z;
  int64_t x_stride, delta_stride, z_stride;
  const void *B, *C_;
  int64_t b_stride, c_stride;
  const float *A, *D, *dbias;
  void *out;
  StateRows init, fin;
  // tiles of L tokens and what a pass leaves for the next one
  int32_t L, ntiles, empties;
  int32_t nseg;   // segments of the tokens that workgroups walk along (k12_scan_walk.hip)
  float *bc;      // [T][G][2][NS] B and C in fp32, padded with zeros
  float *chunk;   // [ntiles][N][C] first each tile's own state, then the state before it
                  // (the walk: that alone, where the caller wants it)
  float *span;    // [ntiles][C] sum of the step sizes over which a state crosses the tile
  float *start;   // [ntiles][N][C] initial state of the last sequence that starts in the tile
  int32_t *flag;  // [ntiles] a sequence starts in the tile
  float *a2;      // [NS][C] log2(e) A, padded with zeros
  // backward
  const void *dy;
  int64_t dy_stride;
  const float *dfin;
  void *dx, *ddelta, *dz, *dB, *dC;
  float *dA, *dD, *ddbias, *dinit;
  float *bct;     // [G][2][NS][Tp] B and C by state, Tp = tokens in whole tiles
  float *gchunk;  // [ntiles][N][C] gradient of the state behind a tile
  float *gspan;   // [ntiles][C]
  int32_t *gflag; // [ntiles] a sequence ends in the tile
  int64_t Tp;
  float *psum;    // [ntiles][N + 2][C] sums of dA, dD and ddelta_bias over a tile
  float *pbc;     // [ncb][2][NS][Tp] sums of dB and dC over a block of channels
  int32_t vec;    // decode: four states of A, B and C are aligned vectors
  int32_t num_cus;
};

// States of a channel that the kernels are compiled for: N and zeros behind it.
constexpr int scan_states(int n) { return n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64; }

hipError_t launch_scan_prepare(const ScanArgs &a, hipStream_t s);
hipError_t launch_scan_states(const ScanArgs &a, hipStream_t s);
hipError_t launch_scan_chain(const ScanArgs &a, bool backward, hipStream_t s);
hipError_t launch_scan_forward(const ScanArgs &a, hipStream_t s);
hipError_t launch_scan_walk(const ScanArgs &a, hipStream_t s);
hipError_t launch_scan_backward(const ScanArgs &a, hipStream_t s);
hipError_t launch_scan_decode(const ScanArgs &a, hipStream_t s);

struct BeamArgs {
  int32_t B, K, V, M;
  int32_t dtype;
  const void *logits;
  int64_t stride;  // elements from a beam's row to the next
  const float *scores;
  float *out_scores;
  int32_t *parents, *tokens;
  // parts of a row and what each leaves
  int32_t parts, part_len;
  float *best;      // [B K parts][M] logits
  int32_t *where;   // [B K parts][M] their tokens
  float *stat;      // [B K parts][2] largest logit, sum of exponentials relative to it
  int32_t vec;
};

hipError_t launch_beam_select(const BeamArgs &a, hipStream_t s);

constexpr int kReorderPools = 16;  // pools of one launch

struct ReorderArgs {
  int32_t B, K, rows, pools;
  const void *idx;      // [B K]
  const void *parents;  // [B, K]
  void *new_idx;        // [B K]
  int32_t type;
  int32_t *status;
  struct Pool {
    char *p;
    int64_t str[4];  // bytes
    int64_t d2, d3, row;  // elements
    int32_t es, flat, align;
    int32_t units, unit;  // units of a row, elements of one
  } pool[kReorderPools];
};

hipError_t launch_pool_reorder(const ReorderArgs &a, hipStream_t s);

#ifdef __HIPCC__

// ----------------------------------------------------------------- elements

template <typename T, int V>
struct alignas(sizeof(T) * V <= 16 && (V & (V - 1)) == 0 ? sizeof(T) * V : sizeof(T)) Vec {
  T e[V];
};

// V consecutive elements, kept in their type, on an address aligned to their size
// (or to 16 bytes, if they are more).
template <typename T, int V> __device__ __forceinline__ Vec<T, V> load_vec(const T *p) {
  constexpr int Q = sizeof(T) * V <= 16 ? V : 16 / (int)sizeof(T);
  if constexpr (V % Q != 0 || (Q & (Q - 1)) != 0) {  // (an odd number: one by one)
    Vec<T, V> v;
#pragma unroll
    for (int e = 0; e < V; ++e) v.e[e] = p[e];
    return v;
  } else if constexpr (Q == V) {
    return *reinterpret_cast<const Vec<T, V> *>(p);
  } else {
    Vec<T, V> v;
#pragma unroll
    for (int q = 0; q < V; q += Q) {
      const Vec<T, Q> part = *reinterpret_cast<const Vec<T, Q> *>(p + q);
#pragma unroll
      for (int e = 0; e < Q; ++e) v.e[q + e] = part.e[e];
    }
    return v;
  }
}
template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V> &v, float (&o)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = to_f32(v.e[e]);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&o)[V]) {
  constexpr int Q = sizeof(T) * V <= 16 ? V : 16 / (int)sizeof(T);
#pragma unroll
  for (int q = 0; q < V; q += Q) {
    Vec<T, Q> v;
#pragma unroll
    for (int e = 0; e < Q; ++e) v.e[e] = from_f32<T>(o[q + e]);
    *reinterpret_cast<Vec<T, Q> *>(p + q) = v;
  }
}

// V elements at each of R offsets, all loads on their way before the first is
// used; vec: on addresses aligned to their size (or to 16 bytes).
template <typename St, int R, int V>
__device__ __forceinline__ void rows_load(const void *base, bool vec, const int64_t (&off)[R],
                                          float (&o)[R][V]) {
  const St *p = (const St *)base;
  Vec<St, V> raw[R];
  if (V > 1 && vec) {
#pragma unroll
    for (int r = 0; r < R; ++r) raw[r] = load_vec<St, V>(p + off[r]);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < V; ++e) raw[r].e[e] = p[off[r] + e];
  }
#pragma unroll
  for (int r = 0; r < R; ++r) widen(raw[r], o[r]);
}
template <typename St, int R, int V>
__device__ __forceinline__ void rows_store(void *base, bool vec, const int64_t (&off)[R],
                                           const float (&o)[R][V]) {
  St *p = (St *)base;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (V > 1 && vec) {
      constexpr int Q = sizeof(St) * V <= 16 ? V : 16 / (int)sizeof(St);
#pragma unroll
      for (int q = 0; q < V; q += Q) {
        Vec<St, Q> v;
#pragma unroll
        for (int e = 0; e < Q; ++e) v.e[e] = from_f32<St>(o[r][q + e]);
        *reinterpret_cast<Vec<St, Q> *>(p + off[r] + q) = v;
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) p[off[r] + e] = from_f32<St>(o[r][e]);
    }
  }
}

// The same of states of any state dtype.
template <int R, int V>
__device__ __forceinline__ void state_read(const StateRows &s, const int64_t (&off)[R],
                                           float (&o)[R][V]) {
  if (s.dtype == GDN_F32) rows_load<float, R, V>(s.p, s.vec, off, o);
  else if (s.dtype == GDN_BF16) rows_load<bf16, R, V>(s.p, s.vec, off, o);
  else if (s.dtype == GDN_F16) rows_load<f16, R, V>(s.p, s.vec, off, o);
  else if (s.dtype == GDN_FP8_E4M3) rows_load<fp8e4m3, R, V>(s.p, s.vec, off, o);
  else rows_load<fp8e5m2, R, V>(s.p, s.vec, off, o);
}
template <int R, int V>
__device__ __forceinline__ void state_write(const StateRows &s, const int64_t (&off)[R],
                                            const float (&o)[R][V]) {
  if (s.dtype == GDN_F32) rows_store<float, R, V>(s.p, s.vec, off, o);
  else if (s.dtype == GDN_BF16) rows_store<bf16, R, V>(s.p, s.vec, off, o);
  else if (s.dtype == GDN_F16) rows_store<f16, R, V>(s.p, s.vec, off, o);
  else if (s.dtype == GDN_FP8_E4M3) rows_store<fp8e4m3, R, V>(s.p, s.vec, off, o);
  else rows_store<fp8e5m2, R, V>(s.p, s.vec, off, o);
}

// V consecutive fp32 values (vec: aligned).
template <int V> __device__ __forceinline__ void f32_load(const float *p, bool vec, float (&o)[V]) {
  const int64_t off[1] = {0};
  float r[1][V];
  rows_load<float, 1, V>(p, vec, off, r);
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = r[0][e];
}

// State row of sequence i; -1 where its index is out of range.
__device__ __forceinline__ int64_t state_row(const Batch &b, int i) {
  if (!b.sidx) return i;
  const int64_t r = load_index_any(b.sidx, b.sidx_type, i);
  return r >= 0 && r < b.pool_rows ? r : -1;
}

// ---------------------------------------------------------------- functions

constexpr float kLog2E = 1.44269504088896341f;

// 1 / (1 + e^-v): 0 and 1 at the infinities.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2E * v));
}

// ----------------------------------------------------------------- geometry

// Sequences of the 64 tokens from t0 on, as one wave's lanes see them: lane s
// stands for token t0 + s.
struct Block64 {
  unsigned long long first, last, valid;  // tokens that start, end, belong to a sequence
  int seq, pos;                           // this lane's token: sequence and place in it
};

// Sequence i of the batch: first token and length, inside [0, T] whatever the
// workspace holds.  For the whole wave; `pre`: the lanes' sequences of a small
// batch, where the caller holds them.
__device__ __forceinline__ void sequence_of(const Batch &b, int i, int lane, int &bos, int &len,
                                            const SeqLane *pre = nullptr) {
  if (!b.bos) {
    const SeqLane s = pre ? *pre : seq_lane(b.cu, b.cu_type, b.N, b.T, lane);
    bos = __builtin_amdgcn_readlane(s.bos, i);
    len = __builtin_amdgcn_readlane(s.len, i);
    return;
  }
  bos = min(max(b.bos[i], 0), (int)b.T);
  len = max(min(b.bos[i + 1], (int)b.T) - bos, 0);
}

// The status word of a small batch, by one wave (larger ones: with bos).
__device__ __forceinline__ void batch_status(const Batch &b, int lane) {
  const SeqLane s = seq_lane(b.cu, b.cu_type, b.N, b.T, lane);
  unsigned bits = 0;
  const long long prev = __shfl_up((long long)s.raw, 1);
  if (b.cu && lane <= b.N && (s.raw < 0 || s.raw > b.T || (lane > 0 && s.raw < prev)))
    bits |= GDN_STATUS_CU_SEQLENS;
  if (b.sidx && lane < b.N && state_row(b, lane) < 0) bits |= GDN_STATUS_STATE_INDEX;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) bits |= __shfl_xor(bits, o);
  if (lane == 0) b.status[0] = (int32_t)bits;
}

// The status word of a decode step, by one workgroup of 256 threads.
__device__ __forceinline__ void decode_status(const Batch &b) {
  __shared__ unsigned bits;
  if (threadIdx.x == 0) bits = 0u;
  __syncthreads();
  if (b.sidx)
    for (int i = threadIdx.x; i < b.N; i += 256)
      if (state_row(b, i) < 0) atomicOr(&bits, GDN_STATUS_STATE_INDEX);
  __syncthreads();
  if (threadIdx.x == 0) b.status[0] = (int32_t)bits;
}

// LDS words written by some lanes of a wave are there for the others.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// `mark`: 64 words of LDS of this wave's own.  Every lane calls it; `pre` as above.
__device__ __forceinline__ Block64 block_geometry(const Batch &b, int t0, int lane, int *mark,
                                                  const SeqLane *pre = nullptr) {
  Block64 g;
  mark[lane] = -1;
  wave_sync();
  int covering;  // the sequence of token t0, if an earlier token starts it
  SeqLane s;
  if (!b.bos) {
    s = pre ? *pre : seq_lane(b.cu, b.cu_type, b.N, b.T, lane);
    const bool some = lane < b.N && s.len > 0;
    const unsigned long long m = __ballot(some && s.bos < t0 && s.bos + s.len > t0);
    covering = m ? 63 - __builtin_clzll(m) : -1;
    if (some && s.bos >= t0 && s.bos < t0 + 64) mark[s.bos - t0] = lane;
  } else {
    // entries of bos at or before t0, in steps of 64
    int lo = 0, n = b.N + 1;
    while (n > 64) {
      const int step = (n + 63) / 64, i = lo + lane * step;
      const int p = __builtin_popcountll(__ballot(i < lo + n && b.bos[min(i, b.N)] <= t0));
      if (p == 0) {
        n = 0;
        break;
      }
      const int end = lo + n;
      lo += (p - 1) * step;
      n = min(step, end - lo);
    }
    lo += __builtin_popcountll(__ballot(lane < n && b.bos[min(lo + lane, b.N)] <= t0)) - 1;
    covering = lo >= 0 && lo < b.N && b.bos[lo] < t0 ? lo : -1;
    for (int base = max(lo, 0); base < b.N; base += 64) {
      const int j = base + lane;
      const int at = b.bos[min(j, b.N)], next = b.bos[min(j + 1, b.N)];
      if (j < b.N && at >= t0 && at < t0 + 64 && next > at) mark[at - t0] = j;
      if (__ballot(j >= b.N || at >= t0 + 64)) break;
    }
  }
  wave_sync();
  int v = mark[lane];
  g.first = __ballot(v >= 0);
  if (lane == 0 && v < 0) v = covering;
  g.seq = wave_prefix_max_nonneg(v + 1) - 1;
  int bos, len;
  if (!b.bos) {
    bos = __shfl(s.bos, max(g.seq, 0));
    len = __shfl(s.len, max(g.seq, 0));
  } else {
    const int i = max(g.seq, 0);
    bos = b.N > 0 ? b.bos[i] : 0;
    len = b.N > 0 ? b.bos[i + 1] - bos : 0;
  }
  g.pos = max(t0 + lane - bos, 0);
  const bool valid = g.seq >= 0 && g.pos < len && t0 + lane < b.T;
  g.valid = __ballot(valid);
  g.last = __ballot(valid && g.pos == len - 1);
  g.first &= g.valid;
  wave_sync();  // mark can be used again
  return g;
}

#endif

}  // namespace gdn
