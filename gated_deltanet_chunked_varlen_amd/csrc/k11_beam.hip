// k11_beam.hip -- beam search over state pools: selection of the best
// continuations, and the rows of state pools brought in the order of the
// selected parents.
//
// Selection.  Continuation v of beam k scores score_k + logit_kv - log sum_v
// exp(logit_kv); the M best of a group's K V are wanted, ties to the lowest
// (beam, token).  Within a beam the order is that of the logits, so the first
// kernel reads every row once, cut into parts: a workgroup keeps its part in
// registers, sums the exponentials relative to the part's largest logit, and
// finds the part's M largest (logit, token) keys.  The smallest of the largest
// logits of 16 (or 64) groups of threads is a bound that at least 16 (64) logits
// reach, usually some 50 of 8192, which are ranked by counting; where more than
// kPass reach it (ties, masked rows) the bound is taken from whole keys, which
// are all different: at most M threads hold one at or above the M-th largest of
// the threads' largest.  The second kernel, a workgroup per group, joins the sums
// (in fp64: scores of different beams are compared) and takes the M best of the
// parts' candidates in the same way.
// Bounded by the vector ALU and HBM for a batch (64 groups of 8 beams, 131 072 tokens
// in bf16: rows 49 us, 2.7 TB/s, 102 when all keys were ranked; the groups 11, 25
// before), by latency for one request (6 and 8.9 us).  4096 logits a workgroup take
// 57 us and 16 384 63, where 8192 took 49.  With 99.9 % of the tokens masked most parts
// have no finite bound, and the batch takes 128 us instead of 57.
//
// Reordering.  Within a group the first child of a parent keeps its row; the
// other children take the rows of beams without a child, in order, and only
// those are copied.  A row is never both source and destination, so nothing has
// to be set aside: one kernel, in which every workgroup works out its group's
// plan from the parents (a wave, by ballots).  Bounded by HBM: 16 groups of 8 beams,
// rows of 1 MB, 20 us for 92 MB; 32 pools of two kinds in one call 4.7 TB/s.  Rows that
// are no whole groups of 16 bytes move an element a lane: 1.1 TB/s in bf16.
#include "gdn_layers.h"

#include <algorithm>

#pragma clang fp contract(off)

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxM = GDN_BEAM_MAX;  // candidates of a group, beams of a group
constexpr float kInf = __builtin_inff();

typedef unsigned long long u64;

// A key orders by value first and by place (ascending) second; none is 0.
__device__ __forceinline__ u64 key_of(float v, unsigned place) {
  const unsigned b = __float_as_uint(v + 0.f);  // -0 is 0
  const unsigned o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (u64)o << 32 | (0xFFFFFFFFu - place);
}
__device__ __forceinline__ float key_value(u64 k) {
  const unsigned o = (unsigned)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ unsigned key_place(u64 k) { return 0xFFFFFFFFu - (unsigned)k; }

// The M largest of the workgroup's keys, E per thread (Key{}: none), sorted into
// `best` (LDS, M entries, Key{} behind the last one).
template <typename Key, int E, int M> struct Largest {
  static constexpr int kKeys = M * E < kThreads ? kThreads : M * E;
  Key top[kThreads];
  Key cand[kKeys];
  Key best[M];
  unsigned count;
  Key bound;

  __device__ __forceinline__ void find(const Key (&k)[E], int m) {
    const int tid = threadIdx.x;
    Key mine{};
#pragma unroll
    for (int e = 0; e < E; ++e) if (k[e] > mine) mine = k[e];
    top[tid] = mine;
    if (tid < M) best[tid] = Key{};
    if (tid == 0) {
      count = 0;
      bound = Key{};
    }
    __syncthreads();
    // this thread's rank among the largest keys (keys are distinct but for Key{})
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < kThreads; ++i) rank += top[i] > mine;
    if (rank == m - 1 && mine > Key{}) bound = mine;
    __syncthreads();
    const Key from = bound;
    if (!(from > mine)) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (!(from > k[e]) && k[e] > Key{}) cand[atomicAdd(&count, 1u)] = k[e];
    }
    __syncthreads();
    const int n = (int)count;
    for (int i = tid; i < n; i += kThreads) {
      const Key x = cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += cand[j] > x;
      if (r < m) best[r] = x;
    }
    __syncthreads();
  }
};

// Candidates that pass a bound, ranked by counting; more of them are left to
// Largest.
constexpr int kPass = 512;

// Lanes of one of the groups whose largest keys' smallest one is the bound: at
// least M groups of the workgroup's 256 threads, so that at least M keys reach it.
constexpr int group_lanes(int M) { return M <= 16 ? 16 : 4; }

// Reductions by lane moves within rows of 16 lanes (all of them receive the
// result), then over the wave's four rows: through LDS each step took as long as
// reading a part of a row does.
template <int CTRL> __device__ __forceinline__ unsigned moved(unsigned x) {
  return (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}
template <int CTRL> __device__ __forceinline__ float moved(float x) {
  return __uint_as_float(moved<CTRL>(__float_as_uint(x)));
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ unsigned larger(unsigned a, unsigned b) { return max(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ unsigned smaller(unsigned a, unsigned b) { return min(a, b); }
__device__ __forceinline__ float of_lane(float x, int l) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), l));
}
__device__ __forceinline__ unsigned of_lane(unsigned x, int l) {
  return (unsigned)__builtin_amdgcn_readlane((int)x, l);
}

// The largest value of the wave and the smallest one of its groups' largest.
template <int M, typename T>
__device__ __forceinline__ void top_and_low(T x, T &top, T &low) {
  T g = larger(x, moved<0xB1>(x));  // quads
  g = larger(g, moved<0x4E>(g));
  T hi = larger(g, moved<0x124>(g)), lo = smaller(g, moved<0x124>(g));
  hi = larger(hi, moved<0x128>(hi));
  lo = group_lanes(M) == 16 ? hi : smaller(lo, moved<0x128>(lo));
  top = larger(larger(of_lane(hi, 0), of_lane(hi, 16)), larger(of_lane(hi, 32), of_lane(hi, 48)));
  low = smaller(smaller(of_lane(lo, 0), of_lane(lo, 16)),
                smaller(of_lane(lo, 32), of_lane(lo, 48)));
}
__device__ __forceinline__ float wave_max(float x) {
  float top, low;
  top_and_low<16>(x, top, low);
  return top;
}
// A sum over the wave: rows in fp32, their sums in fp64.
__device__ __forceinline__ double wave_sum(float x) {
  x += moved<0xB1>(x);
  x += moved<0x4E>(x);
  x += moved<0x124>(x);
  x += moved<0x128>(x);
  return ((double)of_lane(x, 0) + (double)of_lane(x, 16)) +
         ((double)of_lane(x, 32) + (double)of_lane(x, 48));
}
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

template <typename Key> struct Pass {
  Key key[kPass];
  unsigned count;
};

// A part of one row, E logits per thread.  VEC: rows are whole aligned groups of
// 16 bytes.
template <typename T, int E, int M, bool VEC>
__global__ void __launch_bounds__(kThreads) beam_rows_kernel(BeamArgs a) {
  constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
  constexpr int S = E / V;  // vectors per thread
  constexpr int kWaves = kThreads / 64;
  __shared__ union {
    Largest<u64, E, M> all;
    Pass<u64> pass;
  } L;
  __shared__ float s_top[kWaves], s_low[kWaves];
  __shared__ double s_sum[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const int from = part * a.part_len, to = min(from + a.part_len, a.V);
  const int64_t o = (int64_t)blockIdx.x;
  if (!(a.scores[row] > -kInf)) {
    // a beam that has ended: its continuations are all alike
    if (tid < a.M) {
      a.best[o * a.M + tid] = -kInf;
      a.where[o * a.M + tid] = from + tid < to ? from + tid : -1;
    }
    if (tid == 0) {
      a.stat[2 * o] = -kInf;
      a.stat[2 * o + 1] = 0.f;
    }
    return;
  }
  const T *p = (const T *)a.logits + (int64_t)row * a.stride;
  float x[E];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int at = from + (s * kThreads + tid) * V;
    float v[V];
    if (at < to) {
      widen(load_vec<T, V>(p + at), v);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = -kInf;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) x[s * V + e] = fmaxf(v[e], -kInf);  // NaN: never taken
  }
  if (tid == 0) L.pass.count = 0;
  float mine = -kInf;
#pragma unroll
  for (int e = 0; e < E; ++e) mine = fmaxf(mine, x[e]);
  float of_wave, low;
  top_and_low<M>(mine, of_wave, low);
  if (lane == 0) {
    s_top[wave] = of_wave;
    s_low[wave] = low;
  }
  __syncthreads();
  const float top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  const float bound = fminf(fminf(s_low[0], s_low[1]), fminf(s_low[2], s_low[3]));
  // sum of exponentials relative to the largest logit (of infinite ones each
  // counts 1, and nothing else does)
  float sum = 0.f;
  if (fabsf(top) < kInf) {
#pragma unroll
    for (int e = 0; e < E; ++e) sum += __builtin_amdgcn_exp2f(kLog2E * (x[e] - top));
  } else if (top > 0.f) {
#pragma unroll
    for (int e = 0; e < E; ++e) sum += x[e] == top ? 1.f : 0.f;
  }
  const double all = wave_sum(sum);
  if (lane == 0) s_sum[wave] = all;
  auto place = [&](int k) { return from + (k / V * kThreads + tid) * V + k % V; };
  auto pass = [&](int e) {
    const unsigned at = atomicAdd(&L.pass.count, 1u);
    if (at < kPass) L.pass.key[at] = key_of(x[e], (unsigned)place(e));
  };
  if (bound > -kInf) {
    // few of them, so that most registers are passed over by the whole wave
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (__ballot(x[e] >= bound) != 0 && x[e] >= bound) pass(e);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (place(e) < to) pass(e);
  }
  __syncthreads();
  const int n = (int)L.pass.count;
  if (tid == 0) {
    a.stat[2 * o] = top;
    a.stat[2 * o + 1] = (float)((s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]));
  }
  auto put = [&](int r, u64 b) {
    a.best[o * a.M + r] = b ? key_value(b) : -kInf;
    a.where[o * a.M + r] = b ? (int)key_place(b) : -1;
  };
  if (n <= kPass) {
    for (int i = tid; i < n; i += kThreads) {
      const u64 k = L.pass.key[i];
      int r = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) r += L.pass.key[j] > k;
      if (r < a.M) put(r, k);
    }
    if (tid >= n && tid < a.M) put(tid, 0);  // fewer tokens than places
    return;
  }
  __syncthreads();
  u64 k[E];
#pragma unroll
  for (int e = 0; e < E; ++e) k[e] = place(e) < to ? key_of(x[e], (unsigned)place(e)) : 0;
  L.all.find(k, a.M);
  if (tid < a.M) put(tid, L.all.best[tid]);
}

// A score in fp64, in the order of whole numbers, and (beam, token) descending; the
// lowest bit of place is 0 where unequal logits may have this score.
struct Score {
  u64 value, place;
  __device__ __forceinline__ bool operator>(const Score &o) const {
    return value > o.value || (value == o.value && place > o.place);
  }
};
__device__ __forceinline__ u64 order_of(double v) {
  const u64 b = (u64)__double_as_longlong(v + 0.0);
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double value_of(u64 o) {
  return __longlong_as_double((long long)(o >> 63 ? o & ~(1ull << 63) : ~o));
}

constexpr int kTake = 8;  // candidates per thread and round
constexpr int kScan = 8;  // vectors per thread and round of a look at whole rows

// The first of 2^32 keys for which a condition holds that holds for all behind it too
// (of those from lo on, n of them; lo + n: none), by the whole wave.
template <typename F>
__device__ __forceinline__ unsigned first_key(unsigned lo, unsigned n, F holds) {
  const int lane = threadIdx.x & 63;
  while (n > 0) {
    const unsigned step = (n + 63) / 64;
    const int p = __builtin_popcountll(
        __ballot((u64)lane * step < n && !holds(lo + (unsigned)lane * step)));
    if (p == 0) break;
    const unsigned to = (unsigned)(p - 1) * step + 1;
    lo += to;
    n = min(step - 1, n - to);
  }
  return lo;
}

// Which logits of a round, from token `from` on, are in [low, high]: bit s V + e stands
// for token from + (256 s + thread) V + e.
template <typename T, int V>
__device__ __forceinline__ u64 matches_of(const BeamArgs &a, int64_t row, int from, float low,
                                          float high) {
  const T *p = (const T *)a.logits + row;
  const int first = from + (int)threadIdx.x * V;
  Vec<T, V> raw[kScan];
#pragma unroll
  for (int s = 0; s < kScan; ++s) {
    const int at = first + s * kThreads * V;
    raw[s] = load_vec<T, V>(p + (at < a.V ? at : 0));
  }
  u64 found = 0;
#pragma unroll
  for (int s = 0; s < kScan; ++s) {
    float x[V];
    widen(raw[s], x);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float v = fmaxf(x[e], -kInf);
      if (first + s * kThreads * V < a.V && v >= low && v <= high) found |= 1ull << (s * V + e);
    }
  }
  return found;
}

// One group.  Candidates come in rounds of kTake a thread; those of a round that
// reach its bound, with the best so far, are ranked by counting.
//
// A beam's candidates are its largest logits, and their scores are in the same
// order, but not strictly: where |score|, |largest logit| or |log| is so large that
// 64 bits do not tell unequal logits' scores apart, or infinite, a token that is no
// candidate can have the last place's score and stand before it.  Such scores carry
// a mark, and if the last place's has it, the places of its score are filled again
// from whole rows (64 groups of 8 beams of 131 072 tokens, one candidate of logit 0: 75
// us, 56 for another; 237 when every logit's score was formed).
template <int M> __global__ void __launch_bounds__(kThreads) beam_group_kernel(BeamArgs a) {
  constexpr int kWaves = kThreads / 64;
  __shared__ union {
    Largest<Score, kTake + 1, M> all;
    Pass<Score> pass;
  } L;
  __shared__ Score s_best[M];
  __shared__ double s_log[kMaxM];
  __shared__ unsigned s_low[kWaves];
  __shared__ float s_top[kMaxM], s_score[kMaxM];
  __shared__ int s_count[kWaves];
  __shared__ unsigned s_any;
  __shared__ u64 s_beams;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x;
  const int per = a.parts * a.M, n = a.K * per;
  const int64_t first = (int64_t)b * a.K * a.parts;
  // the first round's candidates are on their way while the sums are joined
  int at[kTake];
  float logit[kTake];
  auto fetch = [&](int base) {
#pragma unroll
    for (int e = 0; e < kTake; ++e) {
      const int i = base + e * kThreads + tid;
      at[e] = i < n ? a.where[first * a.M + i] : -1;
      logit[e] = i < n ? a.best[first * a.M + i] : 0.f;
    }
  };
  fetch(0);
  for (int k = wave; k < a.K; k += kWaves) {
    const float *st = a.stat + 2 * (first + (int64_t)k * a.parts);
    const float score = a.scores[(int64_t)b * a.K + k];
    float top = -kInf, own = lane < a.parts ? st[2 * lane] : -kInf;
    const float part = lane < a.parts ? st[2 * lane + 1] : 0.f;
    for (int i = lane; i < a.parts; i += 64) top = fmaxf(top, st[2 * i]);
    top = wave_max(top);
    double sum = own == top ? (double)part : (double)part * exp((double)own - (double)top);
    for (int i = lane + 64; i < a.parts; i += 64) {
      own = st[2 * i];
      sum += own == top ? (double)st[2 * i + 1]
                        : (double)st[2 * i + 1] * exp((double)own - (double)top);
    }
    sum = wave_sum(sum);
    if (lane == 0) {
      s_top[k] = top;
      s_score[k] = score;
      s_log[k] = log(sum);
    }
  }
  if (tid < M) s_best[tid] = Score{};
  __syncthreads();
  // (of an infinite largest logit the others have no share)
  auto score_at = [&](int k, float logit) {
    const float score = s_score[k], top = s_top[k];
    if (!(logit > -kInf && score > -kInf)) return -(double)kInf;
    const double own = logit == top ? 0.0 : (double)logit - (double)top;
    return own > -(double)kInf ? (double)score + (own - s_log[k]) : -(double)kInf;
  };
  // Whether another logit of beam k may have the same score: the next one is 2^-24
  // of |logit| away at least, and the three sums' roundings, of at most `most`, come
  // to less than 2^-50 of it for both.
  auto may_tie = [&](int k, float logit) {
    const float score = s_score[k], top = s_top[k];
    if (!(score > -kInf)) return false;  // all of its tokens are alike
    if (!(logit > -kInf)) return top == kInf;
    const float most = fabsf(score) + fabsf(top) + fabsf(logit) + fabsf((float)s_log[k]);
    return !(fabsf(logit) > most * 0x1p-26f);
  };
  for (int base = 0; base < n; base += kTake * kThreads) {
    Score c[kTake + 1];
    if (base > 0) fetch(base);
    c[kTake] = tid < a.M ? s_best[tid] : Score{};  // the best so far, one a thread
    const Score last = s_best[a.M - 1];
    bool any = base == 0;
    u64 mine = c[kTake].value;
#pragma unroll
    for (int e = 0; e < kTake; ++e) {
      const int i = base + e * kThreads + tid;
      c[e] = Score{};
      if (at[e] < 0) continue;
      const int k = i / per;
      const u64 flat = (u64)k * (u64)a.V + (u64)at[e];
      const u64 mark = may_tie(k, logit[e]) ? 1 : 0;
      c[e] = Score{order_of(score_at(k, logit[e])), ~(flat << 1 | mark)};
      any |= c[e] > last;
      mine = c[e].value > mine ? c[e].value : mine;
    }
    // nothing better than what there is: on to the next ones
    if (!__syncthreads_or(any)) continue;
    // (the bound: the upper half of a score's order)
    unsigned top, low;
    top_and_low<M>((unsigned)(mine >> 32), top, low);
    if (lane == 0) s_low[wave] = low;
    if (tid == 0) L.pass.count = 0;
    __syncthreads();
    unsigned low32 = s_low[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) low32 = min(low32, s_low[w]);
    const u64 bound = low32 > 0 ? (u64)low32 << 32 : 1;
    if (mine >= bound) {
#pragma unroll
      for (int e = 0; e <= kTake; ++e)
        if (c[e].value >= bound) {
          const unsigned slot = atomicAdd(&L.pass.count, 1u);
          if (slot < kPass) L.pass.key[slot] = c[e];
        }
    }
    __syncthreads();
    const int m = (int)L.pass.count;
    if (m <= kPass) {
      Score keep[2];
      int rank[2] = {M, M};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int i = tid + q * kThreads;
        if (i >= m) continue;
        keep[q] = L.pass.key[i];
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < m; ++j) r += L.pass.key[j] > keep[q];
        rank[q] = r;
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (rank[q] < a.M) s_best[rank[q]] = keep[q];
    } else {
      __syncthreads();
      L.all.find(c, a.M);
      if (tid < a.M) s_best[tid] = L.all.best[tid];
    }
    __syncthreads();
  }
  const Score last = s_best[a.M - 1];
  if (!(last.place & 1)) {
    // Of the beams that have a candidate in one of these places (a part that leaves out
    // a token of this score leaves M candidates, the last of this score too), up to the
    // last place's token.
    const int V = !a.vec ? 1 : a.dtype == GDN_F32 ? 4 : 8;
    const u64 behind = (~last.place >> 1) + 1;
    if (tid == 0) {
      s_beams = 0;
      s_any = 0;
    }
    __syncthreads();
    int have = 0;  // places that are filled: better scores, then the tokens found
    for (int i = 0; i < a.M; ++i) have += s_best[i].value > last.value;
    if (tid >= have && tid < a.M)
      atomicOr(&s_beams, 1ull << (int)((~s_best[tid].place >> 1) / (u64)a.V));
    __syncthreads();
    for (int k = 0; k < a.K && have < a.M; ++k) {
      if (!(s_beams >> k & 1)) continue;
      const int64_t row = ((int64_t)b * a.K + k) * a.stride;
      const u64 flat = (u64)k * (u64)a.V;
      const int end = (int)min((u64)a.V, behind - flat);
      // a beam's scores rise with its logits: those of this score are a range
      constexpr unsigned kLow = 0x007FFFFFu, kHigh = 0xFF800000u;  // keys of -inf and +inf
      auto score_of = [&](unsigned key) {
        return order_of(score_at(k, key_value((u64)key << 32)));
      };
      const unsigned low_key = first_key(kLow, kHigh - kLow + 1, [&](unsigned key) {
        return score_of(key) >= last.value;
      });
      const unsigned next_key = first_key(low_key, kHigh - low_key + 1, [&](unsigned key) {
        return score_of(key) > last.value;
      });
      if (next_key <= low_key) continue;
      const float low = key_value((u64)low_key << 32), high = key_value((u64)(next_key - 1) << 32);
      for (int from = 0; from < end && have < a.M; from += kScan * kThreads * V) {
        const u64 found =
            a.dtype == GDN_F32    ? a.vec ? matches_of<float, 4>(a, row, from, low, high)
                                          : matches_of<float, 1>(a, row, from, low, high)
            : a.dtype == GDN_BF16 ? a.vec ? matches_of<bf16, 8>(a, row, from, low, high)
                                          : matches_of<bf16, 1>(a, row, from, low, high)
                                  : a.vec ? matches_of<f16, 8>(a, row, from, low, high)
                                          : matches_of<f16, 1>(a, row, from, low, high);
        if (!__syncthreads_or(found != 0)) continue;
        const u64 vector = (1ull << V) - 1;
        unsigned mine = 0;
        for (int s = 0; s < kScan; ++s) mine |= (found >> (s * V) & vector) != 0 ? 1u << s : 0u;
        if (mine != 0) atomicOr(&s_any, mine);
        __syncthreads();
        for (unsigned any = s_any; any != 0 && have < a.M; any &= any - 1) {
          const int s = __builtin_ctz(any);
          u64 here = found >> (s * V) & vector;
          const int own = __builtin_popcountll(here), sum = wave_prefix_sum_i(own);
          if (lane == 63) s_count[wave] = sum;
          __syncthreads();
          int place = have + sum - own;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            if (w < wave) place += s_count[w];
            have += s_count[w];
          }
          for (; here != 0 && place < a.M; here &= here - 1, ++place) {
            const int t = from + (s * kThreads + tid) * V + __builtin_ctzll(here);
            s_best[place] = Score{last.value, ~((flat + (u64)t) << 1)};
          }
          __syncthreads();
        }
        if (tid == 0) s_any = 0;  // (set again behind the next round's barrier)
      }
    }
  }
  if (tid >= a.M) return;
  const Score best = s_best[tid];
  const u64 flat = ~best.place >> 1;
  const int64_t o = (int64_t)b * a.M + tid;
  a.out_scores[o] = (float)value_of(best.value);
  a.parents[o] = (int)(flat / (u64)a.V);
  a.tokens[o] = (int)(flat % (u64)a.V);
}

// -------------------------------------------------------------------- reorder

// Child j's share of its group's plan: the beam whose old row it takes, and the
// parent if that row has to be overwritten with its row (else -1).
struct Share {
  int row_of, from;
};

// For the whole wave; parents of the group, one a lane.
__device__ __forceinline__ Share share_of(int parent, int K, int j) {
  u64 used = 0, first = 0;
  for (int i = 0; i < K; ++i) {
    const int q = __builtin_amdgcn_readlane(parent, i);
    if ((unsigned)q < (unsigned)K && !(used >> q & 1)) {
      used |= 1ull << q;
      first |= 1ull << i;
    }
  }
  const int own = __builtin_amdgcn_readlane(parent, j);
  if (first >> j & 1) return {own, -1};
  // of the children that keep no row the r-th takes the r-th row that is left
  const u64 all = K < 64 ? (1ull << K) - 1 : ~0ull;
  u64 left = ~used & all;
  for (int r = __builtin_popcountll(~first & ((1ull << j) - 1)); r > 0; --r) left &= left - 1;
  return {__builtin_ctzll(left), (unsigned)own < (unsigned)K ? own : -1};
}

// The status word, by a workgroup of its own.
__device__ __forceinline__ void reorder_status(const ReorderArgs &a, unsigned *map) {
  __shared__ unsigned s_bits;
  const int words = (a.rows + 31) / 32;
  for (int i = threadIdx.x; i < words; i += kThreads) map[i] = 0u;
  if (threadIdx.x == 0) s_bits = 0u;
  __syncthreads();
  unsigned bits = 0;
  for (int64_t i = threadIdx.x; i < (int64_t)a.B * a.K; i += kThreads) {
    const int64_t r = load_index_any(a.idx, a.type, i), p = load_index_any(a.parents, a.type, i);
    if (p < -1 || p >= a.K || r < -1 || r >= a.rows) bits |= GDN_STATUS_POOL_ROW;
    if (r >= 0 && r < a.rows && (atomicOr(&map[r >> 5], 1u << (r & 31)) >> (r & 31) & 1))
      bits |= GDN_STATUS_POOL_DUPLICATE;
  }
  if (bits) atomicOr(&s_bits, bits);
  __syncthreads();
  if (threadIdx.x == 0) a.status[0] = (int32_t)s_bits;
}

template <typename V>
__device__ __forceinline__ void copy_bytes(const char *src, char *dst, int64_t b0, int64_t b1) {
  constexpr int U = 4;
  constexpr int64_t step = (int64_t)sizeof(V) * kThreads;
  for (int64_t b = b0 + (int64_t)sizeof(V) * threadIdx.x; b < b1; b += U * step) {
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (b + u * step < b1) v[u] = *(const V *)(src + b + u * step);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (b + u * step < b1) *(V *)(dst + b + u * step) = v[u];
  }
}

template <typename U>
__device__ __forceinline__ void copy_strided(const ReorderArgs::Pool &p, const char *src, char *dst,
                                             int64_t e0, int64_t e1) {
  for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) {
    const int64_t k = e % p.d3, r = e / p.d3;
    const int64_t off = (r / p.d2) * p.str[1] + (r % p.d2) * p.str[2] + k * p.str[3];
    *(U *)(dst + off) = *(const U *)(src + off);
  }
}

__global__ void __launch_bounds__(kThreads) pool_reorder_kernel(ReorderArgs a) {
  extern __shared__ unsigned map[];
  const ReorderArgs::Pool &p = a.pool[blockIdx.y];
  const int64_t unit = blockIdx.x, beam = unit / p.units;
  if (beam >= (int64_t)a.B * a.K) {
    if (a.status && blockIdx.y == 0 && blockIdx.x == gridDim.x - 1) reorder_status(a, map);
    return;
  }
  const int lane = threadIdx.x & 63, j = (int)(beam % a.K);
  const int64_t group = beam - j;
  int parent = -1;
  if (lane < a.K) {
    const int64_t q = load_index_any(a.parents, a.type, group + lane);
    parent = q >= 0 && q < a.K ? (int)q : -1;
  }
  const Share s = share_of(parent, a.K, j);
  const int64_t to = load_index_any(a.idx, a.type, group + s.row_of);
  const int slice = (int)(unit % p.units);
  if (a.new_idx && blockIdx.y == 0 && slice == 0 && threadIdx.x == 0) {
    if (a.type == GDN_I64) ((int64_t *)a.new_idx)[beam] = to;
    else ((int32_t *)a.new_idx)[beam] = (int32_t)to;
  }
  if (s.from < 0) return;
  const int64_t from = load_index_any(a.idx, a.type, group + s.from);
  if (to < 0 || to >= a.rows || from < 0 || from >= a.rows || from == to) return;
  const char *src = p.p + from * p.str[0];
  char *dst = p.p + to * p.str[0];
  const int64_t e0 = (int64_t)slice * p.unit, e1 = min(e0 + p.unit, p.row);
  if (p.flat) {
    if (p.align >= 16) copy_bytes<u32x4>(src, dst, e0 * p.es, e1 * p.es);
    else if (p.es == 4) copy_bytes<uint32_t>(src, dst, e0 * 4, e1 * 4);
    else if (p.es == 2) copy_bytes<uint16_t>(src, dst, e0 * 2, e1 * 2);
    else copy_bytes<uint8_t>(src, dst, e0, e1);
  } else if (p.es == 4) {
    copy_strided<uint32_t>(p, src, dst, e0, e1);
  } else if (p.es == 2) {
    copy_strided<uint16_t>(p, src, dst, e0, e1);
  } else {
    copy_strided<uint8_t>(p, src, dst, e0, e1);
  }
}

// ------------------------------------------------------------------- launches

template <typename T, int E, int M> hipError_t rows(const BeamArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.B * a.K * a.parts)), block(kThreads);
  if (a.vec) beam_rows_kernel<T, E, M, true><<<grid, block, 0, s>>>(a);
  else beam_rows_kernel<T, E, M, false><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}
template <typename T> hipError_t rows_of(const BeamArgs &a, hipStream_t s) {
  if (a.part_len > 8 * kThreads)
    return a.M <= 16 ? rows<T, 32, 16>(a, s) : rows<T, 32, kMaxM>(a, s);
  return a.M <= 16 ? rows<T, 8, 16>(a, s) : rows<T, 8, kMaxM>(a, s);
}

}  // namespace

hipError_t launch_beam_select(const BeamArgs &a, hipStream_t s) {
  const hipError_t e = a.dtype == GDN_F32    ? rows_of<float>(a, s)
                       : a.dtype == GDN_BF16 ? rows_of<bf16>(a, s)
                                             : rows_of<f16>(a, s);
  if (e != hipSuccess) return e;
  if (a.M <= 16) beam_group_kernel<16><<<dim3(a.B), dim3(kThreads), 0, s>>>(a);
  else beam_group_kernel<kMaxM><<<dim3(a.B), dim3(kThreads), 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_pool_reorder(const ReorderArgs &a, hipStream_t s) {
  int64_t units = 0;
  for (int i = 0; i < a.pools; ++i) units = std::max<int64_t>(units, a.pool[i].units);
  units *= (int64_t)a.B * a.K;
  const unsigned x = (unsigned)units + (a.status ? 1u : 0u);
  if (x == 0) return hipSuccess;
  const int lds = a.status ? (a.rows + 31) / 32 * 4 : 0;
  pool_reorder_kernel<<<dim3(x, (unsigned)a.pools), dim3(kThreads), lds, s>>>(a);
  return hipGetLastError();
}

}  // namespace gdn
