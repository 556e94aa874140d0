// k6_recurrence.hip -- the gated linear recurrence h_t = g_t h_{t-1} + x_t:
// forward scan, backward scan and decode step.
//
// A tile is 64 tokens x 256 channels, one workgroup of eight waves: wave w
// holds tokens 8 w .. 8 w + 7 of all 256 channels in registers, four channels
// per lane, so that x and g are read from memory once.  Over a run of tokens
// the recurrence is the affine map h -> A h + B (A the product of the gates, B
// the run's last state from zero), and maps compose, so a tile takes
//   1. each wave: its (A, B), from registers                       (sweep 1)
//   2. one thread per channel: the tile's (A, B) from the waves' (LDS), the
//      state before the tile, each wave's start state
//   3. each wave: the true states from its start, written out      (sweep 2)
// The state before a tile comes through the chain: every tile publishes its
// (A, B) as soon as it has it, and its last state once it knows it.  A tile
// looks back over up to kWindow earlier tiles for the nearest last state and
// applies the (A, B) of the tiles between, oldest first.  Every tile forms its
// own last state as fma(A, start, B) too, so the arithmetic is the same
// wherever the looking back ends: results do not depend on timing.
//
// Chain words.  One 64-bit word per tile and channel, written and read by
// relaxed atomics of device scope, carries its own state, so no fence is
// needed: high half kPending (not published), kLast (low half = last state)
// or A (low half = B).  Both marks are NaN patterns that A never takes (a NaN
// A is stored as the default NaN).
// Progress.  Workgroups take tiles in the order of a ticket counter, earlier
// tiles of a channel block first.  A tile waits only for tiles with smaller
// tickets, which were taken by workgroups that are already running; the
// smallest unfinished ticket waits for nothing, so every wait ends.
//
// Sequence bounds.  A token that starts a sequence folds its initial state
// into x (x + g h0) and takes no h from the left; the carry is selected, not
// multiplied by zero, so a NaN or infinity of one sequence never reaches the
// next.  The backward scan runs the chain from the last tile to the first,
// with the carry c_t = g_t dh_t.
#include "gdn_common.h"
#include "gdn_internal.h"
#include "gdn_recurrence.h"

// Products and sums are contracted only where fmaf says so: every variant of a
// kernel then does the same arithmetic.
#pragma clang fp contract(off)

namespace gdn {

namespace {

constexpr int kTok = 8;                     // tokens per wave
constexpr int kWaves = kRecTile / kTok;     // waves per workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kWindow = 16;                 // tiles looked back over
constexpr unsigned kPending = 0xFFFFFFFFu, kLast = 0xFFFFFFFEu;

typedef float f32x4v __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ memory access

// Four consecutive elements as fp32; `left` of them exist (VEC: all four, on
// an address aligned to their size).
template <typename T, bool VEC>
__device__ __forceinline__ void load4(const T *p, int left, float (&o)[4]) {
  if (VEC) {
    typedef T vec __attribute__((ext_vector_type(4)));
    const vec v = *reinterpret_cast<const vec *>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = to_f32((T)v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = e < left ? to_f32(p[e]) : 0.f;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store4(T *p, int left, const float (&o)[4]) {
  if (VEC) {
    typedef T vec __attribute__((ext_vector_type(4)));
    const f32x4v f = {o[0], o[1], o[2], o[3]};
    *reinterpret_cast<vec *>(p) = __builtin_convertvector(f, vec);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) p[e] = from_f32<T>(o[e]);
  }
}

template <typename St>
__device__ __forceinline__ void state_load(const void *base, int64_t off, int left,
                                           float (&o)[4]) {
  const St *p = (const St *)base + off;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = e < left ? to_f32(p[e]) : 0.f;
}
template <typename St>
__device__ __forceinline__ void state_store(void *base, int64_t off, int left,
                                            const float (&o)[4]) {
  St *p = (St *)base + off;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) p[e] = from_f32<St>(o[e]);
}

// Four channels of a state row of any state dtype.  Rows may start anywhere;
// an fp32 row group on a 16-byte boundary moves as one vector.
__device__ __forceinline__ void load_state(const void *base, int dtype, int64_t off, int left,
                                           float (&o)[4]) {
  if (dtype == GDN_F32) {
    const float *p = (const float *)base + off;
    if (left >= 4 && ((uintptr_t)p & 15) == 0) {
      const f32x4v v = *reinterpret_cast<const f32x4v *>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = v[e];
    } else {
      state_load<float>(base, off, left, o);
    }
  } else if (dtype == GDN_BF16) state_load<bf16>(base, off, left, o);
  else if (dtype == GDN_F16) state_load<f16>(base, off, left, o);
  else if (dtype == GDN_FP8_E4M3) state_load<fp8e4m3>(base, off, left, o);
  else state_load<fp8e5m2>(base, off, left, o);
}
__device__ __forceinline__ void store_state(void *base, int dtype, int64_t off, int left,
                                            const float (&o)[4]) {
  if (dtype == GDN_F32) {
    float *p = (float *)base + off;
    if (left >= 4 && ((uintptr_t)p & 15) == 0) {
      const f32x4v v = {o[0], o[1], o[2], o[3]};
      *reinterpret_cast<f32x4v *>(p) = v;
    } else {
      state_store<float>(base, off, left, o);
    }
  } else if (dtype == GDN_BF16) state_store<bf16>(base, off, left, o);
  else if (dtype == GDN_F16) state_store<f16>(base, off, left, o);
  else if (dtype == GDN_FP8_E4M3) state_store<fp8e4m3>(base, off, left, o);
  else state_store<fp8e5m2>(base, off, left, o);
}

// State row of sequence i; -1 where its index is out of range.
__device__ __forceinline__ int64_t state_row(const RecArgs &a, int i) {
  if (!a.sidx) return i;
  const int64_t r = load_index_any(a.sidx, a.sidx_type, i);
  return r >= 0 && r < a.pool_rows ? r : -1;
}

// Initial state of sequence i, channels c .. c + left - 1 (zero without one).
__device__ __forceinline__ void load_init(const RecArgs &a, int i, int c, int left,
                                          float (&o)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = 0.f;
  if (!a.init) return;
  const int64_t r = state_row(a, i);
  if (r >= 0) load_state(a.init, a.init_dtype, r * a.init_stride + c, left, o);
}
__device__ __forceinline__ void store_final(const RecArgs &a, int i, int c, int left,
                                            const float (&o)[4]) {
  const int64_t r = state_row(a, i);
  if (r >= 0) store_state(a.fin, a.fin_dtype, r * a.fin_stride + c, left, o);
}

// -------------------------------------------------------------------- chain

__device__ __forceinline__ void publish(unsigned long long *w, unsigned hi, float lo) {
  __hip_atomic_store(w, ((unsigned long long)hi << 32) | __float_as_uint(lo), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned map_bits(float A) {
  return A != A ? 0x7FC00000u : __float_as_uint(A);
}

// Value carried into `tile` from its neighbour at tile + step, for one
// channel; avail >= 1 tiles lie in that direction, and the last of them always
// publishes kLast by itself.
__device__ __forceinline__ float look_back(const unsigned long long *words, int64_t C, int tile,
                                           int c, int step, int avail) {
  const unsigned long long *base = words + (int64_t)tile * C + c;
  const int64_t d = (int64_t)step * C;
  for (;;) {
    unsigned long long w[kWindow];
    int found = -1;
    bool open = true;  // every nearer tile has published
#pragma unroll
    for (int j0 = 0; j0 < kWindow; j0 += 4) {
      if (found < 0 && open && j0 < avail) {
#pragma unroll
        for (int j = j0; j < j0 + 4; ++j)
          w[j] = j < avail ? __hip_atomic_load(base + (int64_t)(j + 1) * d, __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT)
                           : (unsigned long long)kPending << 32;
#pragma unroll
        for (int j = j0; j < j0 + 4; ++j) {
          const unsigned hi = (unsigned)(w[j] >> 32);
          if (found < 0 && open) {
            if (hi == kLast) found = j;
            else if (hi == kPending) open = false;
          }
        }
      }
    }
    if (found >= 0) {
      float h = 0.f;
#pragma unroll
      for (int j = kWindow - 1; j >= 0; --j) {
        const float lo = __uint_as_float((unsigned)w[j]);
        const float A = __uint_as_float((unsigned)(w[j] >> 32));
        if (j == found) h = lo;
        else if (j < found) h = fmaf(A, h, lo);
      }
      return h;
    }
    __builtin_amdgcn_s_sleep(2);
  }
}

// ----------------------------------------------------------------- geometry

struct TileGeo {
  int lo, hi;             // tokens that belong to a sequence
  int start[kRecTile];    // sequence that starts at this token of the tile, or -1
  int end[kRecTile];      // sequence that ends with it, or -1
};

// Marks of the tile that starts at token t0, by the whole workgroup.  The
// first tile's channel block 0 of a small batch writes the status word.
__device__ __forceinline__ void tile_geometry(const RecArgs &a, int t0, bool status_unit,
                                              TileGeo &G) {
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid < kRecTile) G.start[tid] = G.end[tid] = -1;
  __syncthreads();
  const int t1 = t0 + kRecTile;
  if (!a.bos) {
    if (tid < 64) {
      const SeqLane s = seq_lane(a.cu, a.cu_type, a.N, a.T, lane);
      if (lane < a.N && s.len > 0) {
        if (s.bos >= t0 && s.bos < t1) G.start[s.bos - t0] = lane;
        const int e = s.bos + s.len - 1;
        if (e >= t0 && e < t1) G.end[e - t0] = lane;
      }
      if (lane == 0) G.lo = s.bos;
      if (lane == a.N) G.hi = s.bos;
      if (status_unit && a.status) {
        unsigned bits = 0;
        const long long prev = __shfl_up((long long)s.raw, 1);
        if (a.cu && lane <= a.N && (s.raw < 0 || s.raw > a.T || (lane > 0 && s.raw < prev)))
          bits |= GDN_STATUS_CU_SEQLENS;
        if (a.sidx && lane < a.N && state_row(a, lane) < 0) bits |= GDN_STATUS_STATE_INDEX;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) bits |= __shfl_xor(bits, o);
        if (lane == 0) a.status[0] = (int32_t)bits;
      }
    }
  } else {
    // first j with bos[j] >= t0, then every start and end inside the tile
    int lo = 0, hi = a.N + 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.bos[mid] >= t0) hi = mid; else lo = mid + 1;
    }
    for (int base = lo; base <= a.N && a.bos[base] <= t1; base += kThreads) {
      const int j = base + tid;
      if (j <= a.N) {
        const int b = a.bos[j];
        if (b < t1 && j < a.N && a.bos[j + 1] > b) G.start[b - t0] = j;
        if (b > t0 && b <= t1 && j > 0 && a.bos[j - 1] < b) G.end[b - 1 - t0] = j - 1;
      }
    }
    if (tid == 0) {
      G.lo = a.bos[0];
      G.hi = a.bos[a.N];
    }
  }
  __syncthreads();
}

// Calls f(i) for every empty sequence, spread over the workgroup's waves (i
// is the same for all lanes of a wave).
template <typename F>
__device__ __forceinline__ void for_empty_sequences(const RecArgs &a, F f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (!a.bos) {
    if (wave != 0) return;
    const SeqLane s = seq_lane(a.cu, a.cu_type, a.N, a.T, lane);
    unsigned long long m = __ballot(lane < a.N && s.len == 0);
    for (; m; m &= m - 1) f(__ffsll((long long)m) - 1);
    return;
  }
  for (int base = 64 * wave; base < a.N; base += kThreads) {
    const int i = base + lane;
    unsigned long long m = __ballot(i < a.N && a.bos[i] == a.bos[i + 1]);
    for (; m; m &= m - 1) f(base + __ffsll((long long)m) - 1);
  }
}

// The unit this workgroup works on next: a ticket, or its block index.
__device__ __forceinline__ unsigned next_unit(const RecArgs &a, unsigned &sh) {
  if (!a.ticket) return blockIdx.x;
  __syncthreads();  // LDS of the unit before is free, and so is sh
  if (threadIdx.x == 0)
    sh = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return sh;
}

// Gate of token row t for a lane's four channels (PH: their head's).
template <typename Tg, bool PH, bool VEC>
__device__ __forceinline__ void load_gate(const RecArgs &a, int64_t t, int c, int left, int head,
                                          float (&g)[PH ? 1 : 4]) {
  const Tg *p = (const Tg *)a.g + t * a.g_stride;
  if constexpr (PH) g[0] = to_f32(p[head]);
  else load4<Tg, VEC>(p + c, left, g);
}

// The marked tokens' values of v (wave-uniform `at`), for a lane's channels.
__device__ __forceinline__ void pick(const float (&v)[kTok][4], int at, float (&o)[4]) {
#pragma unroll
  for (int s = 0; s < kTok; ++s)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = s == at || s == 0 ? v[s][e] : o[e];
}

// x + g h0 at the tokens of `first`.
template <bool PH>
__device__ __forceinline__ void fold_initial(const RecArgs &a, unsigned first, int id, int c,
                                             int left, const float (&g)[kTok][PH ? 1 : 4],
                                             float (&x)[kTok][4]) {
  for (unsigned m = first; m; m &= m - 1) {
    const int at = __builtin_ctz(m);
    float h0[4];
    load_init(a, __builtin_amdgcn_readlane(id, at), c, left, h0);
#pragma unroll
    for (int s = 0; s < kTok; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[s][e] = s == at ? fmaf(g[s][PH ? 0 : e], h0[e], x[s][e]) : x[s][e];
  }
}

// ------------------------------------------------------------------ forward

// Bounded by HBM: per element x and g are read once and out written once; the
// chain adds 8 bytes per tile and channel each for clearing, publishing twice
// and looking back.
template <typename Tx, typename Tg, bool PH, bool VEC>
__global__ void __launch_bounds__(kThreads) rec_forward_kernel(RecArgs a) {
  constexpr int GV = PH ? 1 : 4;
  __shared__ TileGeo G;
  __shared__ float sA[kWaves][kRecChannels], sB[kWaves][kRecChannels];
  __shared__ int s_reset[kWaves];
  __shared__ unsigned s_unit;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (;;) {
    const unsigned u = next_unit(a, s_unit);
    if (u >= a.units) return;
    const int tile = (int)(u / (unsigned)a.ncb), cb = (int)(u % (unsigned)a.ncb);
    const int t0 = tile * kRecTile, tw = t0 + wave * kTok;
    const int c = cb * kRecChannels + 4 * lane;
    const int left = min(4, a.C - c);
    const int head = PH ? min(c, a.C - 1) / a.D : 0;

    float x[kTok][4], g[kTok][GV];
#pragma unroll
    for (int s = 0; s < kTok; ++s) {
      const int64_t t = tw + s;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[s][e] = 0.f;
#pragma unroll
      for (int e = 0; e < GV; ++e) g[s][e] = 1.f;
      if (t < a.T && left > 0) {
        load4<Tx, VEC>((const Tx *)a.x + t * a.x_stride + c, left, x[s]);
        load_gate<Tg, PH, VEC>(a, t, c, left, head, g[s]);
      }
    }
    tile_geometry(a, t0, u == 0, G);

    // marks of this wave's tokens, as wave-uniform bits
    const int my = wave * kTok + (lane & (kTok - 1));
    const int id_s = G.start[my], id_e = G.end[my];
    const unsigned first = (unsigned)__ballot(id_s >= 0) & ((1u << kTok) - 1);
    const unsigned last = (unsigned)__ballot(id_e >= 0) & ((1u << kTok) - 1);
    const int glo = G.lo, ghi = G.hi;

    // tokens outside every sequence: the identity
#pragma unroll
    for (int s = 0; s < kTok; ++s) {
      if (tw + s < glo || tw + s >= ghi) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[s][e] = 0.f;
#pragma unroll
        for (int e = 0; e < GV; ++e) g[s][e] = 1.f;
      }
    }
    if (a.init) fold_initial<PH>(a, first, id_s, c, left, g, x);
    {
      float A[4] = {1.f, 1.f, 1.f, 1.f}, B[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < kTok; ++s) {
        const bool st = first >> s & 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float gg = g[s][PH ? 0 : e];
          B[e] = st ? x[s][e] : fmaf(gg, B[e], x[s][e]);
          A[e] *= gg;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sA[wave][4 * lane + e] = A[e];
        sB[wave][4 * lane + e] = B[e];
      }
      if (lane == 0) s_reset[wave] = first != 0;
    }
    __syncthreads();

    if (tid < kRecChannels) {
      const int ch = cb * kRecChannels + tid;
      if (ch < a.C) {
        float A = 1.f, B = 0.f, h = 0.f;
        bool reset = tile == 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const bool r = s_reset[w];
          B = r ? sB[w][tid] : fmaf(sA[w][tid], B, sB[w][tid]);
          A *= sA[w][tid];
          reset |= r;
        }
        if (a.ticket) {
          unsigned long long *w = a.words + (int64_t)tile * a.C + ch;
          if (reset) publish(w, kLast, B);
          else publish(w, map_bits(A), B);
          if (tile > 0) {
            h = look_back(a.words, a.C, tile, ch, -1, tile);
            if (!reset) publish(w, kLast, fmaf(A, h, B));
          }
        }
        if (a.chunk) a.chunk[(int64_t)tile * a.C + ch] = h;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float b = sB[w][tid], aa = sA[w][tid];
          sB[w][tid] = h;
          h = s_reset[w] ? b : fmaf(aa, h, b);
        }
      }
    }
    __syncthreads();

    if (left > 0) {
      float h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = sB[wave][4 * lane + e];
#pragma unroll
      for (int s = 0; s < kTok; ++s) {
        const int64_t t = tw + s;
        const bool st = first >> s & 1;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h[e] = st ? x[s][e] : fmaf(g[s][PH ? 0 : e], h[e], x[s][e]);
        if (a.out && t >= glo && t < ghi) store4<Tx, VEC>((Tx *)a.out + t * a.C + c, left, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[s][e] = h[e];
      }
      if (a.fin) {
        for (unsigned m = last; m; m &= m - 1) {
          const int at = __builtin_ctz(m);
          pick(x, at, h);
          store_final(a, __builtin_amdgcn_readlane(id_e, at), c, left, h);
        }
      }
    }
    if (tile == 0 && a.fin) {
      for_empty_sequences(a, [&](int i) {
        float h0[4];
        load_init(a, i, c, left, h0);
        if (left > 0) store_final(a, i, c, left, h0);
      });
    }
    if (!a.ticket) return;
  }
}

// ----------------------------------------------------------------- backward

// One pass over x, g and dy: the states before each token are formed again
// from the tile's saved start state, in fp32, while the carry of the gradient
// comes through the chain from the tiles behind.  Bounded by HBM.
template <typename Tx, typename Tg, bool PH, bool VEC>
__global__ void __launch_bounds__(kThreads) rec_backward_kernel(RecArgs a) {
  constexpr int GV = PH ? 1 : 4;
  __shared__ TileGeo G;
  __shared__ float sA[kWaves][kRecChannels], sF[kWaves][kRecChannels], sB[kWaves][kRecChannels];
  __shared__ int s_first[kWaves], s_last[kWaves];
  __shared__ unsigned s_unit;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (;;) {
    const unsigned u = next_unit(a, s_unit);
    if (u >= a.units) return;
    const int tile = a.ntiles - 1 - (int)(u / (unsigned)a.ncb), cb = (int)(u % (unsigned)a.ncb);
    const int t0 = tile * kRecTile, tw = t0 + wave * kTok;
    const int c = cb * kRecChannels + 4 * lane;
    const int left = min(4, a.C - c);
    const int head = PH ? min(c, a.C - 1) / a.D : 0;

    float x[kTok][4], g[kTok][GV], dy[kTok][4];
#pragma unroll
    for (int s = 0; s < kTok; ++s) {
      const int64_t t = tw + s;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[s][e] = dy[s][e] = 0.f;
#pragma unroll
      for (int e = 0; e < GV; ++e) g[s][e] = 1.f;
      if (t < a.T && left > 0) {
        load4<Tx, VEC>((const Tx *)a.x + t * a.x_stride + c, left, x[s]);
        load4<Tx, VEC>((const Tx *)a.dy + t * a.dy_stride + c, left, dy[s]);
        load_gate<Tg, PH, VEC>(a, t, c, left, head, g[s]);
      }
    }
    tile_geometry(a, t0, u == 0, G);

    const int my = wave * kTok + (lane & (kTok - 1));
    const int id_s = G.start[my], id_e = G.end[my];
    const unsigned first = (unsigned)__ballot(id_s >= 0) & ((1u << kTok) - 1);
    const unsigned last = (unsigned)__ballot(id_e >= 0) & ((1u << kTok) - 1);
    const int glo = G.lo, ghi = G.hi;
#pragma unroll
    for (int s = 0; s < kTok; ++s) {
      if (tw + s < glo || tw + s >= ghi) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[s][e] = dy[s][e] = 0.f;
#pragma unroll
        for (int e = 0; e < GV; ++e) g[s][e] = 1.f;
      }
    }
    if (a.init) fold_initial<PH>(a, first, id_s, c, left, g, x);
    if (a.dfin) {
      for (unsigned m = last; m; m &= m - 1) {
        const int at = __builtin_ctz(m);
        float d[4];
        load_state(a.dfin, GDN_F32, (int64_t)__builtin_amdgcn_readlane(id_e, at) * a.C + c, left,
                   d);
#pragma unroll
        for (int s = 0; s < kTok; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) dy[s][e] += s == at ? d[e] : 0.f;
      }
    }
    {
      float A[4] = {1.f, 1.f, 1.f, 1.f}, F[4] = {0.f, 0.f, 0.f, 0.f}, B[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < kTok; ++s) {
        const bool st = first >> s & 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float gg = g[s][PH ? 0 : e];
          F[e] = st ? x[s][e] : fmaf(gg, F[e], x[s][e]);
          A[e] *= gg;
        }
      }
#pragma unroll
      for (int s = kTok - 1; s >= 0; --s) {
        const bool en = last >> s & 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) B[e] = g[s][PH ? 0 : e] * (en ? dy[s][e] : dy[s][e] + B[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sA[wave][4 * lane + e] = A[e];
        sF[wave][4 * lane + e] = F[e];
        sB[wave][4 * lane + e] = B[e];
      }
      if (lane == 0) {
        s_first[wave] = first != 0;
        s_last[wave] = last != 0;
      }
    }
    __syncthreads();

    if (tid < kRecChannels) {
      const int ch = cb * kRecChannels + tid;
      if (ch < a.C) {
        float A = 1.f, B = 0.f, k = 0.f;
        bool reset = tile == a.ntiles - 1;
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w) {
          const bool r = s_last[w];
          B = r ? sB[w][tid] : fmaf(sA[w][tid], B, sB[w][tid]);
          A *= sA[w][tid];
          reset |= r;
        }
        if (a.ticket) {
          unsigned long long *w = a.words + (int64_t)tile * a.C + ch;
          if (reset) publish(w, kLast, B);
          else publish(w, map_bits(A), B);
          if (tile < a.ntiles - 1) {
            k = look_back(a.words, a.C, tile, ch, 1, a.ntiles - 1 - tile);
            if (!reset) publish(w, kLast, fmaf(A, k, B));
          }
        }
        float h = a.chunk ? a.chunk[(int64_t)tile * a.C + ch] : 0.f;
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w) {
          const float b = sB[w][tid];
          sB[w][tid] = k;
          k = s_last[w] ? b : fmaf(sA[w][tid], k, b);
        }
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = sF[w][tid];
          sF[w][tid] = h;
          h = s_first[w] ? f : fmaf(sA[w][tid], h, f);
        }
      }
    }
    __syncthreads();

    if (left > 0) {
      // x becomes the state before each token
      float h[4], k[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[e] = sF[wave][4 * lane + e];
        k[e] = sB[wave][4 * lane + e];
      }
#pragma unroll
      for (int s = 0; s < kTok; ++s) {
        const bool st = first >> s & 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float now = st ? x[s][e] : fmaf(g[s][PH ? 0 : e], h[e], x[s][e]);
          x[s][e] = st ? 0.f : h[e];
          h[e] = now;
        }
      }
      if (a.init) {
        for (unsigned m = first; m; m &= m - 1) {
          const int at = __builtin_ctz(m);
          float h0[4];
          load_init(a, __builtin_amdgcn_readlane(id_s, at), c, left, h0);
#pragma unroll
          for (int s = 0; s < kTok; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[s][e] = s == at ? h0[e] : x[s][e];
        }
      }
#pragma unroll
      for (int s = kTok - 1; s >= 0; --s) {
        const int64_t t = tw + s;
        const bool en = last >> s & 1;
        const bool inside = t >= glo && t < ghi;
        float dh[4], dg[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dh[e] = en ? dy[s][e] : dy[s][e] + k[e];
          dg[e] = inside ? dh[e] * x[s][e] : 0.f;
          k[e] = g[s][PH ? 0 : e] * dh[e];
          if (!inside) dh[e] = 0.f;
        }
        if constexpr (PH) {
          // a head's D / 4 lanes (8, 16 or 32) lie next to each other
          float sum = (dg[0] + dg[1]) + (dg[2] + dg[3]);
          for (int o = 1; o < a.D / 4; o <<= 1) sum += __shfl_xor(sum, o);
          if (t < a.T && (c % a.D) == 0)
            ((Tg *)a.dg)[t * a.H + head] = from_f32<Tg>(sum);
        } else if (t < a.T) {
          store4<Tg, VEC>((Tg *)a.dg + t * a.C + c, left, dg);
        }
        if (t < a.T) store4<Tx, VEC>((Tx *)a.dx + t * a.C + c, left, dh);
#pragma unroll
        for (int e = 0; e < 4; ++e) dy[s][e] = k[e];  // the carry out of this token
      }
      if (a.dinit) {
        for (unsigned m = first; m; m &= m - 1) {
          const int at = __builtin_ctz(m);
          pick(dy, at, k);
          store_state(a.dinit, GDN_F32, (int64_t)__builtin_amdgcn_readlane(id_s, at) * a.C + c,
                      left, k);
        }
      }
    }
    if (tile == 0 && a.dinit) {
      for_empty_sequences(a, [&](int i) {
        if (left > 0) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          if (a.dfin) load_state(a.dfin, GDN_F32, (int64_t)i * a.C + c, left, d);
          store_state(a.dinit, GDN_F32, (int64_t)i * a.C + c, left, d);
        }
      });
    }
    if (!a.ticket) return;
  }
}

// ------------------------------------------------------------------- decode

// One thread per four channels of one sequence: the state row is read,
// updated and written back.  Bounded by launch latency below a few hundred
// sequences, by HBM above.
template <typename Tx, typename Tg, bool PH, bool VEC>
__global__ void __launch_bounds__(256) rec_decode_kernel(RecArgs a) {
  if (blockIdx.x == 0 && a.status) {
    __shared__ unsigned bits;
    if (threadIdx.x == 0) bits = 0u;
    __syncthreads();
    if (a.sidx)
      for (int i = threadIdx.x; i < a.N; i += 256)
        if (state_row(a, i) < 0) atomicOr(&bits, GDN_STATUS_STATE_INDEX);
    __syncthreads();
    if (threadIdx.x == 0) a.status[0] = (int32_t)bits;
  }
  const int per = (a.C + 3) / 4;  // threads of one sequence
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)per * a.N) return;
  const int i = (int)(id / per), c = 4 * (int)(id % per);
  const int left = min(4, a.C - c);
  float x[4], g[PH ? 1 : 4], h[4];
  load4<Tx, VEC>((const Tx *)a.x + i * a.x_stride + c, left, x);
  load_gate<Tg, PH, VEC>(a, i, c, left, PH ? c / a.D : 0, g);
  load_init(a, i, c, left, h);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = fmaf(g[PH ? 0 : e], h[e], x[e]);
  store4<Tx, VEC>((Tx *)a.out + (int64_t)i * a.C + c, left, h);
  if (a.fin) store_final(a, i, c, left, h);
}

// ------------------------------------------------------------------ prepare

constexpr int kPrepThreads = 1024;

// Chain words to kPending and the ticket to zero; block 0 of a large batch
// also forms the sanitised sequence starts (running maximum of cu_seqlens
// clamped to [0, T]) and the status word.
__global__ void __launch_bounds__(kPrepThreads) rec_prepare_kernel(RecArgs a, int32_t *bos) {
  const int tid = threadIdx.x;
  if (a.ticket) {
    const int64_t n = (int64_t)a.ntiles * a.C;
    for (int64_t i = (int64_t)blockIdx.x * kPrepThreads + tid; i < n;
         i += (int64_t)gridDim.x * kPrepThreads)
      a.words[i] = ~0ull;
    if (blockIdx.x == 0 && tid == 0) *a.ticket = 0u;
  }
  if (blockIdx.x != 0 || !bos) return;
  __shared__ int s_wave[kPrepThreads / 64];
  __shared__ int s_carry;
  __shared__ unsigned s_bits;
  const int lane = tid & 63, wave = tid >> 6;
  if (tid == 0) {
    s_carry = 0;
    s_bits = 0u;
  }
  __syncthreads();
  for (int64_t base = 0; base <= a.N; base += kPrepThreads) {
    const int64_t i = base + tid;
    int x = 0;
    if (i <= a.N) {
      const int64_t raw = load_index_any(a.cu, a.cu_type, i);
      const int64_t y = raw < 0 ? 0 : (raw > a.T ? a.T : raw);
      bool bad = raw != y;
      if (i > 0) bad |= raw < load_index_any(a.cu, a.cu_type, i - 1);
      if (bad) atomicOr(&s_bits, GDN_STATUS_CU_SEQLENS);
      if (i < a.N && a.sidx && state_row(a, (int)i) < 0)
        atomicOr(&s_bits, GDN_STATUS_STATE_INDEX);
      x = (int)y;
    }
    int m = wave_prefix_max_nonneg(x);
    if (lane == 63) s_wave[wave] = m;
    __syncthreads();
    m = max(m, s_carry);
    for (int w = 0; w < wave; ++w) m = max(m, s_wave[w]);
    if (i <= a.N) bos[i] = m;
    __syncthreads();
    if (tid == kPrepThreads - 1) s_carry = m;
    __syncthreads();
  }
  if (tid == 0 && a.status) a.status[0] = (int32_t)s_bits;
}

// Calls f(kernel tag) for the call's types and layout.
template <template <typename, typename, bool, bool> class L>
hipError_t dispatch(const RecArgs &a, hipStream_t s) {
#define GDN_REC_GO(TX, TG)                                                              \
  return a.g_per_head ? (a.vec ? L<TX, TG, true, true>::go(a, s)                        \
                               : L<TX, TG, true, false>::go(a, s))                      \
                      : (a.vec ? L<TX, TG, false, true>::go(a, s)                       \
                               : L<TX, TG, false, false>::go(a, s))
  if (a.x_dtype == GDN_F32) { GDN_REC_GO(float, float); }
  if (a.x_dtype == GDN_BF16) {
    if (a.g_dtype == GDN_F32) { GDN_REC_GO(bf16, float); }
    GDN_REC_GO(bf16, bf16);
  }
  if (a.g_dtype == GDN_F32) { GDN_REC_GO(f16, float); }
  GDN_REC_GO(f16, f16);
#undef GDN_REC_GO
}

// Workgroups of a scan: one per unit up to 8 per compute unit, which then take
// further tickets.
unsigned scan_grid(const RecArgs &a) {
  const uint32_t most = 8u * (uint32_t)a.num_cus;
  return a.ticket && a.units > most ? most : a.units;
}

template <typename Tx, typename Tg, bool PH, bool VEC> struct Fwd {
  static hipError_t go(const RecArgs &a, hipStream_t s) {
    rec_forward_kernel<Tx, Tg, PH, VEC><<<dim3(scan_grid(a)), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
  }
};
template <typename Tx, typename Tg, bool PH, bool VEC> struct Bwd {
  static hipError_t go(const RecArgs &a, hipStream_t s) {
    rec_backward_kernel<Tx, Tg, PH, VEC><<<dim3(scan_grid(a)), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
  }
};
template <typename Tx, typename Tg, bool PH, bool VEC> struct Dec {
  static hipError_t go(const RecArgs &a, hipStream_t s) {
    const int64_t threads = (int64_t)((a.C + 3) / 4) * a.N;
    const int64_t blocks = threads > 0 ? (threads + 255) / 256 : 1;
    rec_decode_kernel<Tx, Tg, PH, VEC><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(a);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_rec_prepare(const RecArgs &a, int32_t *bos, hipStream_t s) {
  const int64_t n = a.ticket ? (int64_t)a.ntiles * a.C : 1;
  const int64_t want = (n + 4 * kPrepThreads - 1) / (4 * kPrepThreads);
  const int64_t most = 2 * (int64_t)a.num_cus;
  rec_prepare_kernel<<<dim3((unsigned)(want < most ? want : most)), dim3(kPrepThreads), 0, s>>>(
      a, bos);
  return hipGetLastError();
}
hipError_t launch_rec_forward(const RecArgs &a, hipStream_t s) { return dispatch<Fwd>(a, s); }
hipError_t launch_rec_backward(const RecArgs &a, hipStream_t s) { return dispatch<Bwd>(a, s); }
hipError_t launch_rec_decode(const RecArgs &a, hipStream_t s) { return dispatch<Dec>(a, s); }

}  // namespace gdn
