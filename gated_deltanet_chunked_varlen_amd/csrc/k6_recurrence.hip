// k6_recurrence.hip -- the gated linear recurrence h_t = g_t h_{t-1} + x_t:
// forward scan, backward scan and decode step.
//
// A tile is 64 (or 128) tokens x 256 channels, one workgroup of eight waves:
// wave w holds tokens 8 w .. 8 w + 7 (16 w .. 16 w + 15) of all 256 channels in
// registers, four channels per lane, so that x and g are read from memory
// once.  Over a run of tokens the recurrence is the affine map h -> A h + B (A
// the product of the gates, B the run's last state from zero), and maps
// compose, so a tile takes
//   1. each wave: its (A, B), from registers                       (sweep 1)
//   2. one thread per channel: the tile's (A, B) from the waves' (LDS), the
//      state before the tile, each wave's start state
//   3. each wave: the true states from its start, written out      (sweep 2)
// The state before a tile comes through a chain of two levels.  Every tile
// publishes its (A, B) as soon as it has it.  Eight tiles are a group; the last
// tile of a group composes the group's (A, B) from theirs and publishes it
// too, and the group's last state once it knows it.  A tile looks back over up
// to kWindow earlier groups for the nearest last state, applies the (A, B) of
// the groups between, oldest first, and then the composed (A, B) of the tiles
// before it in its own group.  Each step of this arithmetic is fixed by the
// tile's place, wherever the looking back ends, so results do not depend on
// timing.  (One level over eight tiles took 5.4 us of 24 at 2 x 2048 tokens:
// a hop of 1.5 us for every eight tiles, against two hops for 64.)
//
// Chain words.  One 64-bit word per tile (and per group) and channel, written
// and read by relaxed atomics of device scope, carries its own state, so no
// fence is needed: high half kPending (not published), kLast (low half = last
// state, nothing before it matters) or A (low half = B).  Both marks are NaN
// patterns that A never takes (a NaN A is stored as the default NaN).
// Progress.  Each channel block has a ticket counter that hands out its tiles
// in order (one counter for all made 512 workgroups queue for 5 us).  A tile
// waits only for earlier tiles of its channel block, which were taken by
// workgroups that are already running; the first unfinished one waits for
// nothing, so every wait ends.  That needs a workspace that nobody else writes
// during the call.  If one does (two calls at once given the same one), a wait
// gives up after wait_limit looks with a NaN for the state, a ticket behind the
// last tile ends its workgroup, and sequence starts read from the workspace are
// taken only inside the tile: the results are wrong, but the call ends and
// writes nothing but its own buffers.
//
// Sequence bounds.  A wave walks its tokens segment by segment, a segment
// being the wave's part of one sequence; where a sequence starts the carry is
// replaced by its initial state, never multiplied by zero, so a NaN or
// infinity of one sequence does not reach the next.  Within a sequence an
// infinite state stays infinite under gates above 0, so a product of such gates
// that underflows is kept at kTiny (0 * infinity would be NaN).  Sweep 1 needs the last
// segment only (the first one, going backward): what lies before a start does
// not leave the wave.  The backward scan runs the chain from the last tile to
// the first, with the carry k_t = g_t dh_t.
#include "gdn_common.h"
#include "gdn_internal.h"
#include "gdn_recurrence.h"

// Products and sums are contracted only where fmaf says so: every variant of a
// kernel then does the same arithmetic.
#pragma clang fp contract(off)

namespace gdn {

namespace {

constexpr int kWaves = 8;                   // waves per workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kWindow = 8;                  // groups looked back over
constexpr unsigned kPending = 0xFFFFFFFFu, kLast = 0xFFFFFFFEu, kNaN = 0x7FC00000u;

typedef float f32x4v __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ memory access

template <typename T> using V4 = T __attribute__((ext_vector_type(4)));

// Four consecutive elements, kept in their type until they are used (16-bit
// types: two registers instead of four); `left` of them exist (VEC: all four,
// on an address aligned to their size).
template <typename T, bool VEC>
__device__ __forceinline__ V4<T> load4(const T *p, int left) {
  if (VEC) return *reinterpret_cast<const V4<T> *>(p);
  V4<T> v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = e < left ? p[e] : (T)0.f;
  return v;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store4(T *p, int left, const float (&o)[4]) {
  if (VEC) {
    const f32x4v f = {o[0], o[1], o[2], o[3]};
    *reinterpret_cast<V4<T> *>(p) = __builtin_convertvector(f, V4<T>);
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
__device__ __forceinline__ unsigned long long peek(const unsigned long long *w) {
  return __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// True for some lane, which is unusual: the same for the whole wave, so that it is
// a scalar branch.
__device__ __forceinline__ bool rare(bool b) { return __builtin_expect(__ballot(b) != 0, 0); }

// What a product of gates is kept at where it underflows.  Products are formed
// plainly, and a 0 is looked into afterwards: no gate is 0 if no factor is.
constexpr float kTiny = 0x1p-149f;

__device__ __forceinline__ unsigned mark(unsigned long long w) { return (unsigned)(w >> 32); }
__device__ __forceinline__ float low(unsigned long long w) { return __uint_as_float((unsigned)w); }
__device__ __forceinline__ unsigned map_bits(float A) {
  return A != A ? kNaN : __float_as_uint(A);
}

// State behind the group at g, for one channel; `avail` >= 1 groups lie from g
// on in direction step, and the last of them always publishes kLast by itself.
// NaN if `limit` looks did not find it.
__device__ __forceinline__ float look_back(const unsigned long long *groups, int64_t C, int g,
                                           unsigned c, int step, int avail, unsigned limit) {
  groups += (int64_t)g * C;
  const int64_t d = (int64_t)step * C;
  for (unsigned look = 0;; ++look) {
    unsigned long long w[kWindow];
    int found = -1;
    bool open = true;  // every nearer group has published
#pragma unroll
    for (int j0 = 0; j0 < kWindow; j0 += 4) {
      if (found < 0 && open && j0 < avail) {
#pragma unroll
        for (int j = j0; j < j0 + 4; ++j)
          w[j] = j < avail ? peek(groups + (int64_t)j * d + c) : (unsigned long long)kPending << 32;
#pragma unroll
        for (int j = j0; j < j0 + 4; ++j) {
          if (found < 0 && open) {
            if (mark(w[j]) == kLast) found = j;
            else if (mark(w[j]) == kPending) open = false;
          }
        }
      }
    }
    if (found >= 0) {
      float h = 0.f;
#pragma unroll
      for (int j = kWindow - 1; j >= 0; --j) {
        if (j == found) h = low(w[j]);
        else if (j < found) h = fmaf(__uint_as_float(mark(w[j])), h, low(w[j]));
      }
      return h;
    }
    if (look >= limit) return __uint_as_float(kNaN);
    __builtin_amdgcn_s_sleep(2);
  }
}

// No wave's product of gates is 0, for one channel.
__device__ __forceinline__ bool all_above_zero(const float (&sA)[kWaves][kRecChannels], int ch) {
  bool positive = true;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) positive = positive && sA[w][ch] != 0.f;
  return positive;
}

// A composed map h -> A h + B, or (known) the constant B.
struct Map {
  float A, B;
  bool known;
};

// The tile's place in the chain, for one channel: publishes its map (own) and
// returns the state before it.  step -1: the chain runs from tile 0 upward;
// +1: from the last tile downward.
__device__ __forceinline__ float chain(const RecArgs &a, int tile, unsigned c, int step, Map own) {
  const int n = step < 0 ? tile : a.ntiles - 1 - tile;  // place in the chain
  unsigned long long *word = a.words + (int64_t)tile * a.C + c;
  if (own.known) publish(word, kLast, own.B);
  else publish(word, map_bits(own.A), own.B);
  // the tiles before this one in its group, nearest first up to a known state
  const int before = n % kGroup;
  Map m = {1.f, 0.f, false};
  float A = own.A;  // of the tiles before and this one
  if (before > 0) {
    unsigned long long w[kGroup - 1];
    bool open;
    for (unsigned look = 0;; ++look) {
      open = true;
#pragma unroll
      for (int j = 0; j < kGroup - 1; ++j)
        if (j < before) w[j] = peek(word + (int64_t)(j + 1) * step * a.C);
#pragma unroll
      for (int j = 0; j < kGroup - 1; ++j)
        if (j < before && mark(w[j]) == kPending) open = false;
      if (open || look >= a.wait_limit) break;
      __builtin_amdgcn_s_sleep(2);
    }
#pragma unroll
    for (int j = kGroup - 2; j >= 0; --j) {
      if (j < before) {
        if (mark(w[j]) == kLast) {
          m = {0.f, low(w[j]), true};
        } else {
          const float Aj = __uint_as_float(mark(w[j]));
          m.B = fmaf(Aj, m.B, low(w[j]));
          m.A *= Aj;
        }
      }
    }
    A *= m.A;
    if (rare(A == 0.f && !m.known)) {
      bool positive = true;
#pragma unroll
      for (int j = 0; j < kGroup - 1; ++j)
        if (j < before) positive = positive && __uint_as_float(mark(w[j])) != 0.f;
      if (m.A == 0.f && positive) m.A = kTiny;
      if (A == 0.f && m.A != 0.f && own.A != 0.f) A = kTiny;
    }
    if (!open) m = {0.f, __uint_as_float(kNaN), true};  // given up
  }
  const int group = n / kGroup;
  unsigned long long *gword = a.groups + (int64_t)group * a.C + c;
  const bool closes = before == kGroup - 1;
  if (group == 0) m.known = true;  // nothing before: the state is zero
  Map all = {A, fmaf(own.A, m.B, own.B), m.known};
  if (own.known) all = own;
  if (closes) publish(gword, all.known ? kLast : map_bits(all.A), all.B);
  if (m.known) return m.B;
  const float h = look_back(a.groups, a.C, group - 1, c, -1, group, a.wait_limit);
  if (closes && !all.known) publish(gword, kLast, fmaf(all.A, h, all.B));
  return fmaf(m.A, h, m.B);
}

// Values read from LDS before are read again after, instead of being held in
// registers across the wait of the chain.
__device__ __forceinline__ void reread_lds() { asm volatile("" ::: "memory"); }

// x, of which the compiler knows nothing: work on it is done again, not kept.
__device__ __forceinline__ float opaque(float x) {
  asm volatile("" : "+v"(x));
  return x;
}

// ----------------------------------------------------------------- geometry

template <int TOK> struct TileGeo {
  static constexpr int kTile = kWaves * TOK;
  int lo, hi;         // tokens that belong to a sequence
  int start[kTile];   // sequence that starts at this token of the tile, or -1
  int end[kTile];     // sequence that ends with it, or -1
  int first[kWaves];  // each wave's Marks::first and last
  int last[kWaves];
};

// Marks of the tile that starts at token t0, by the whole workgroup.  The
// first tile's channel block 0 of a small batch writes the status word.
template <int TOK>
__device__ __forceinline__ void tile_geometry(const RecArgs &a, int t0, bool status_unit,
                                              TileGeo<TOK> &G) {
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid < G.kTile) G.start[tid] = G.end[tid] = -1;
  __syncthreads();
  const int t1 = t0 + G.kTile;
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
    // first j with bos[j] >= t0, then every start and end inside the tile (and
    // inside the tokens, whatever the workspace holds)
    const int te = min(t1, (int)a.T);
    int lo = 0, hi = a.N + 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.bos[mid] >= t0) hi = mid; else lo = mid + 1;
    }
    for (int base = lo; base <= a.N && a.bos[base] <= te; base += kThreads) {
      const int j = base + tid;
      if (j <= a.N) {
        const int b = a.bos[j];
        if (b >= t0 && b < te && j < a.N && a.bos[j + 1] > b) G.start[b - t0] = j;
        if (b > t0 && b <= te && j > 0 && a.bos[j - 1] < b) G.end[b - 1 - t0] = j - 1;
      }
    }
    if (tid == 0) {
      G.lo = a.bos[0];
      G.hi = min(a.bos[a.N], (int)a.T);
    }
  }
  __syncthreads();
}

// Calls f(i) for the empty sequences, four at a time (i[k] the same for all
// lanes of a wave, -1: none), so that f has four loads on their way: one after
// the other they took 0.6 us each, 90 us for 170 empty ones in a training step.
// A workgroup takes 64 sequences in turn, each wave eight; these workgroups come
// behind the scan's in the grid and have no part in the chain.
template <typename F>
__device__ __forceinline__ void for_empty_sequences(const RecArgs &a, int part, F f) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto work = [&](int base, unsigned m) {
    while (m) {
      int i[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        i[k] = m ? base + __builtin_ctz(m) : -1;
        m &= m - 1;
      }
      f(i);
    }
  };
  if (!a.bos) {
    const SeqLane s = seq_lane(a.cu, a.cu_type, a.N, a.T, lane);
    const unsigned long long m = __ballot(lane < a.N && s.len == 0);
    work(8 * wave, (unsigned)(m >> (8 * wave)) & 0xFFu);
    return;
  }
  for (int base = 8 * (wave + kWaves * part); base < a.N; base += 8 * kWaves * a.empties) {
    const int i = base + (lane & 7);
    work(base, (unsigned)__ballot(i < a.N && a.bos[i] == a.bos[i + 1]) & 0xFFu);
  }
}

// Final states of the empty sequences: their initial states.
__device__ __forceinline__ void empty_forward(const RecArgs &a, int part, int c, int left) {
  for_empty_sequences(a, part, [&](const int(&i)[4]) {
    if (left <= 0) return;
    int64_t row[4];
    float h[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) row[k] = i[k] >= 0 ? state_row(a, i[k]) : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int e = 0; e < 4; ++e) h[k][e] = 0.f;
      if (a.init && row[k] >= 0)
        load_state(a.init, a.init_dtype, row[k] * a.init_stride + c, left, h[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (row[k] >= 0)
        store_state(a.fin, a.fin_dtype, row[k] * a.fin_stride + c, left, h[k]);
  });
}
// Gradients of their initial states: those of their final states.
__device__ __forceinline__ void empty_backward(const RecArgs &a, int part, int c, int left) {
  for_empty_sequences(a, part, [&](const int(&i)[4]) {
    if (left <= 0) return;
    float d[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int e = 0; e < 4; ++e) d[k][e] = 0.f;
      if (i[k] >= 0 && a.dfin) load_state(a.dfin, GDN_F32, (int64_t)i[k] * a.C + c, left, d[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i[k] >= 0) store_state(a.dinit, GDN_F32, (int64_t)i[k] * a.C + c, left, d[k]);
  });
}

// The channel block of this workgroup and its place in the block's chain (-1: a
// ticket behind the last tile, there is nothing to do).  One
// round of workgroups after another starts one block further: workgroups go
// to the eight XCDs in turn, so without the shift a block of a multiple-of-8
// set would stay on one XCD (65 536 tokens x 16 blocks: 486 us against 410).
__device__ __forceinline__ int take_place(const RecArgs &a, int &cb) {
  cb = (int)((blockIdx.x + blockIdx.x / (unsigned)a.ncb) % (unsigned)a.ncb);
  if (!a.ticket) return 0;
  __shared__ int place;
  if (threadIdx.x == 0)
    place = (int)__hip_atomic_fetch_add(a.ticket + cb * kTicketStep, 1u, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const int n = __builtin_amdgcn_readfirstlane(place);
  return (unsigned)n < (unsigned)a.ntiles ? n : -1;
}

// Gates of one token for a lane's four channels: four values, or their head's.
template <typename Tg, bool PH, bool VEC> struct Gate {
  V4<Tg> v;
  __device__ __forceinline__ void load(const Tg *row, int c, int left, int) {
    v = load4<Tg, VEC>(row + c, left);
  }
  __device__ __forceinline__ float operator[](int e) const { return to_f32((Tg)v[e]); }
};
template <typename Tg, bool VEC> struct Gate<Tg, true, VEC> {
  Tg v;
  __device__ __forceinline__ void load(const Tg *row, int, int, int head) { v = row[head]; }
  __device__ __forceinline__ float operator[](int) const { return to_f32(v); }
};

// The marks of a wave's tokens as wave-uniform bits: tokens that start and end
// a sequence, and those that belong to one, [lo, hi).
template <int TOK> struct Marks {
  unsigned first, last;
  int lo, hi;
  const int *start, *end;  // of the wave's tokens, in LDS

  __device__ __forceinline__ void read(TileGeo<TOK> &G, int t0, int wave, int lane) {
    const int base = wave * TOK;
    start = G.start + base;
    end = G.end + base;
    first = (unsigned)__ballot(start[lane & (TOK - 1)] >= 0) & ((1u << TOK) - 1);
    last = (unsigned)__ballot(end[lane & (TOK - 1)] >= 0) & ((1u << TOK) - 1);
    lo = __builtin_amdgcn_readfirstlane(min(max(G.lo - t0 - base, 0), TOK));
    hi = __builtin_amdgcn_readfirstlane(min(max(G.hi - t0 - base, 0), TOK));
    if (lane == 0) {
      G.first[wave] = (int)first;
      G.last[wave] = (int)last;
    }
  }
  // no sequence starts or ends here, and every token belongs to one
  __device__ __forceinline__ bool plain() const {
    return (first | last) == 0 && lo == 0 && hi == TOK;
  }
  // the wave's last token that starts a sequence
  __device__ __forceinline__ int last_first() const { return 31 - __builtin_clz(first); }
  // sequence that starts / ends at this wave's token s.  Read from LDS, the same
  // for all lanes, where it is needed: kept one per lane it would have to be read
  // from lanes that have no channels, and a register that the compiler puts aside
  // is brought back for the lanes that do.
  __device__ __forceinline__ int seq_first(int s) const {
    return __builtin_amdgcn_readfirstlane(start[s]);
  }
  __device__ __forceinline__ int seq_last(int s) const {
    return __builtin_amdgcn_readfirstlane(end[s]);
  }
};

// Bit w: wave w of the tile has a mark of this kind (after a barrier).
__device__ __forceinline__ unsigned marked_waves(const int (&marks)[kWaves], int lane) {
  return (unsigned)__ballot(marks[lane & (kWaves - 1)] != 0) & ((1u << kWaves) - 1);
}

// f(s) for the tokens s of [lo, hi), ascending or descending.  The bounds are
// wave-uniform, so the conditions are scalar branches.
template <int TOK, typename F>
__device__ __forceinline__ void ascend(int lo, int hi, F f) {
#pragma unroll
  for (int s = 0; s < TOK; ++s)
    if (s >= lo && s < hi) f(s);
}
template <int TOK, typename F>
__device__ __forceinline__ void descend(int lo, int hi, F f) {
#pragma unroll
  for (int s = TOK - 1; s >= 0; --s)
    if (s >= lo && s < hi) f(s);
}

// Calls f(std::true_type) for a wave whose tokens are all in the middle of one
// sequence, else f(std::false_type): the sweeps of most waves then are straight
// code without a condition (packed batch of 23 060 x 4096 with head gates: half
// of all instructions issued were scalar ones for the marks).
template <int TOK, typename F>
__device__ __forceinline__ void by_marks(const Marks<TOK> &m, F f) {
  if (m.plain()) f(std::true_type{});
  else f(std::false_type{});
}

// The product A of a plain wave's gates, formed by plain multiplications: kTiny
// where it underflowed and no gate is 0.  Only a plain wave's product takes part
// in a state that is used: before a wave with a start, or behind the last end, it
// is replaced or belongs to no token.
template <int TOK, typename GateT>
__device__ __forceinline__ void keep_above_zero(const GateT (&g)[TOK], float (&A)[4]) {
  if (!rare(fminf(fminf(fabsf(A[0]), fabsf(A[1])), fminf(fabsf(A[2]), fabsf(A[3]))) == 0.f)) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    bool positive = A[e] == 0.f;
#pragma unroll
    for (int s = 0; s < TOK; ++s) positive = positive && g[s][e] != 0.f;
    if (positive) A[e] = kTiny;
  }
}

// Sweep 1 of the forward map: the wave's (A, B).  h0 receives the initial state
// of the wave's last sequence start, which sweep 2 must not read again: in a
// pool worked on in place, another wave may have written that sequence's final
// state over it by then.
template <typename Tx, bool PLAIN, int TOK, typename GateT>
__device__ __forceinline__ void forward_map(const RecArgs &a, const Marks<TOK> &m,
                                            const V4<Tx> (&x)[TOK], const GateT (&g)[TOK], int c,
                                            int left, float (&A)[4], float (&B)[4],
                                            float (&h0)[4]) {
  int lo = PLAIN ? 0 : m.lo;
#pragma unroll
  for (int e = 0; e < 4; ++e) h0[e] = 0.f;
  if (!PLAIN && m.first) {
    lo = m.last_first();
    load_init(a, m.seq_first(lo), c, left, h0);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    A[e] = 1.f;
    B[e] = h0[e];
  }
  ascend<TOK>(lo, PLAIN ? TOK : m.hi, [&](int s) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float gg = g[s][e];
      B[e] = fmaf(gg, B[e], to_f32((Tx)x[s][e]));
      A[e] *= gg;
    }
  });
  if (PLAIN) keep_above_zero<TOK>(g, A);
}

// The state before token s, which starts a sequence.  Every start of the wave
// but the last has its sequence end in this wave too, after this read.
template <int TOK>
__device__ __forceinline__ void start_state(const RecArgs &a, const Marks<TOK> &m, int s, int c,
                                            int left, const float (&h0)[4], float (&h)[4]) {
  if (s == m.last_first()) {
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = h0[e];
  } else {
    load_init(a, m.seq_first(s), c, left, h);
  }
}

// f(lo, hi, started): the wave's segments in order, `started` where the first
// token starts a sequence.
template <bool PLAIN, int TOK, typename F>
__device__ __forceinline__ void segments_up(const Marks<TOK> &m, F f) {
  if (PLAIN) return f(0, TOK, false);
  unsigned first = m.first;
  int lo = m.lo;
  bool started = false;
  for (;;) {
    const int hi = first ? __builtin_ctz(first) : m.hi;
    if (hi > lo) f(lo, hi, started);
    if (!first) break;
    first &= first - 1;
    lo = hi;
    started = true;
  }
}
// The same from the last to the first.
template <bool PLAIN, int TOK, typename F>
__device__ __forceinline__ void segments_down(const Marks<TOK> &m, F f) {
  if (PLAIN) return f(0, TOK, false);
  unsigned first = m.first;
  int hi = m.hi;
  while (first) {
    const int lo = 31 - __builtin_clz(first);
    if (hi > lo) f(lo, hi, true);
    first &= ~(1u << lo);
    hi = lo;
  }
  if (hi > m.lo) f(m.lo, hi, false);
}

// ------------------------------------------------------------------ forward

// Tokens per wave: 16 for 16-bit x with head gates, which take few registers,
// else 8.  Twice the bytes per workgroup halve the chain's traffic and its share
// of a tile's time (23 060 tokens x 4096 channels, fp16 with head gates: 104 us
// with 8, 87 with 16).  16-bit gates per channel gain nothing (2 x 2048 x 2048: 17.9 and
// 18.9 us); with fp32 gates or fp32 x 16 tokens would leave one workgroup per CU
// instead of two, and they did not fit the backward pass's registers at all.
template <typename T> constexpr int code() {
  return sizeof(T) == 4 ? GDN_F32 : std::is_same<T, bf16>::value ? GDN_BF16 : GDN_F16;
}
template <typename Tx, bool PH> constexpr int forward_tokens() {
  return rec_forward_tile(code<Tx>(), PH) / kWaves;
}

// Bounded by HBM: per element x and g are read once and out written once; the
// chain adds 8 bytes per tile and channel each for clearing, publishing and
// looking back.  65 536 tokens x 4096 channels, bf16 with fp32 gates: 393 us,
// 5.5 TB/s (a plain copy runs at 4.7 to 5.4 TB/s on the same card).  2 x 2048
// tokens x 2048 channels: 19 us; it is one round of workgroups, whose loads and
// stores hardly overlap.  515 x 2048 in fp32: 10.3 us; the code is 60 KB, and what
// a short call runs of it comes into the instruction cache first (2.5 KB more for
// the infinities' sake cost 0.4 us, a form for plain waves alone half of that).
// Two workgroups per CU (128 registers) are what keeps enough
// bytes on their way: with one, the long pass took 666 us.
template <typename Tx, typename Tg, bool PH, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) rec_forward_kernel(RecArgs a) {
  constexpr int TOK = forward_tokens<Tx, PH>();
  __shared__ TileGeo<TOK> G;
  __shared__ float sA[kWaves][kRecChannels], sB[kWaves][kRecChannels];
  // what is the same for a wave's lanes is kept in scalar registers
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (blockIdx.x >= a.units) {
    const unsigned b = blockIdx.x - a.units;
    const int ec = (int)(b % (unsigned)a.ncb) * kRecChannels + 4 * lane;
    return empty_forward(a, (int)(b / (unsigned)a.ncb), ec, min(4, a.C - ec));
  }
  int cb;
  const int tile = take_place(a, cb);
  if (tile < 0) return;
  const int T = (int)a.T;
  const int t0 = tile * G.kTile, tw = t0 + wave * TOK;
  const int c = cb * kRecChannels + 4 * lane;
  const int left = min(4, a.C - c);
  const int head = PH ? min(c, a.C - 1) / a.D : 0;

  V4<Tx> x[TOK];
  Gate<Tg, PH, VEC> g[TOK];
  if (left > 0) {
#pragma unroll
    for (int s = 0; s < TOK; ++s) {
      if (tw + s < T) {
        const int64_t t = tw + s;
        x[s] = load4<Tx, VEC>((const Tx *)a.x + t * a.x_stride + c, left);
        g[s].load((const Tg *)a.g + t * a.g_stride, c, left, head);
      }
    }
  }
  tile_geometry(a, t0, tile == 0 && cb == 0, G);
  Marks<TOK> m;
  m.read(G, t0, wave, lane);
  float h0[4];
  by_marks(m, [&](auto plain) {
    float A[4], B[4];
    forward_map<Tx, decltype(plain)::value>(a, m, x, g, c, left, A, B, h0);
    *reinterpret_cast<f32x4v *>(&sA[wave][4 * lane]) = f32x4v{A[0], A[1], A[2], A[3]};
    *reinterpret_cast<f32x4v *>(&sB[wave][4 * lane]) = f32x4v{B[0], B[1], B[2], B[3]};
  });
  __syncthreads();

  // (before the branches: every lane of the wave takes part)
  const unsigned resets = marked_waves(G.first, lane);
  if (tid < kRecChannels) {
    const int ch = cb * kRecChannels + tid;
    if (ch < a.C) {
      float A = 1.f, B = 0.f, h = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        B = resets >> w & 1 ? sB[w][tid] : fmaf(sA[w][tid], B, sB[w][tid]);
        A *= sA[w][tid];
      }
      if (rare(A == 0.f) && A == 0.f && all_above_zero(sA, tid)) A = kTiny;
      if (a.ticket) {
        h = chain(a, tile, ch, -1, Map{A, B, resets != 0});
        reread_lds();
      }
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int tb = t0 + w * TOK;
        if (w * TOK % GDN_RECURRENCE_CHUNK == 0 && a.chunk && tb < T)
          a.chunk[(int64_t)(tb / GDN_RECURRENCE_CHUNK) * a.C + ch] = h;
        const float b = sB[w][tid], aa = sA[w][tid];
        sB[w][tid] = h;
        h = resets >> w & 1 ? b : fmaf(aa, h, b);
      }
    }
  }
  __syncthreads();

  if (left > 0) {
    float h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = sB[wave][4 * lane + e];
    by_marks(m, [&](auto plain) {
      constexpr bool P = decltype(plain)::value;
      segments_up<P>(m, [&](int lo, int hi, bool started) {
        if (!P && started) start_state(a, m, lo, c, left, h0, h);
        ascend<TOK>(lo, hi, [&](int s) {
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = fmaf(g[s][e], h[e], to_f32((Tx)x[s][e]));
          if (a.out) store4<Tx, VEC>((Tx *)a.out + (int64_t)(tw + s) * a.C + c, left, h);
        });
        if (!P && a.fin && (m.last >> (hi - 1) & 1))
          store_final(a, m.seq_last(hi - 1), c, left, h);
      });
    });
  }
}

// Sum over a head's D / 4 lanes (8, 16 or 32 next to each other) by lane moves
// within the vector unit: neighbours, pairs, quads and eights of a row of 16
// hold equal sums in turn, and a second row takes the first one's.  The last
// lane of the head has the sum.
__device__ __forceinline__ float head_sum(float x, int D) {
  x += dpp_or_zero<0xB1>(x);   // quad_perm [1, 0, 3, 2]
  x += dpp_or_zero<0x4E>(x);   // quad_perm [2, 3, 0, 1]
  x += dpp_or_zero<0x141>(x);  // row_half_mirror: the other quad of eight
  if (D >= 64) x += dpp_or_zero<0x140>(x);         // row_mirror: the other eight
  if (D >= 128) x += dpp_or_zero<0x142, 0xA>(x);   // row_bcast:15 into rows 1 and 3
  return x;
}

// ----------------------------------------------------------------- backward

// One pass over x, g and dy: the states before each token are formed again
// from the tile's saved start state, in fp32, while the carry of the gradient
// comes through the chain from the tiles behind.  2 x 2048 tokens x 2048
// channels, bf16 with fp32 gates: 26 us, 4.5 TB/s.  23 060 x 4096, fp16 with
// head gates: 154 us, 3.7 TB/s; there the vector units are busy a third of the
// time and a tile's 14 us are split between its loads, some 700 vector
// instructions per wave and the chain.
template <typename Tx, typename Tg, bool PH, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) rec_backward_kernel(RecArgs a) {
  constexpr int TOK = 8;
  __shared__ TileGeo<TOK> G;
  __shared__ float sA[kWaves][kRecChannels], sF[kWaves][kRecChannels], sB[kWaves][kRecChannels];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (blockIdx.x >= a.units) {
    const unsigned b = blockIdx.x - a.units;
    const int ec = (int)(b % (unsigned)a.ncb) * kRecChannels + 4 * lane;
    return empty_backward(a, (int)(b / (unsigned)a.ncb), ec, min(4, a.C - ec));
  }
  int cb;
  const int place = take_place(a, cb);
  if (place < 0) return;
  const int tile = a.ntiles - 1 - place;
  const int T = (int)a.T;
  const int t0 = tile * G.kTile, tw = t0 + wave * TOK;
  const int c = cb * kRecChannels + 4 * lane;
  const int left = min(4, a.C - c);
  const int head = PH ? min(c, a.C - 1) / a.D : 0;

  V4<Tx> x[TOK], dy[TOK];
  Gate<Tg, PH, VEC> g[TOK];
  if (left > 0) {
#pragma unroll
    for (int s = 0; s < TOK; ++s) {
      if (tw + s < T) {
        const int64_t t = tw + s;
        x[s] = load4<Tx, VEC>((const Tx *)a.x + t * a.x_stride + c, left);
        dy[s] = load4<Tx, VEC>((const Tx *)a.dy + t * a.dy_stride + c, left);
        g[s].load((const Tg *)a.g + t * a.g_stride, c, left, head);
      }
    }
  }
  tile_geometry(a, t0, tile == 0 && cb == 0, G);
  Marks<TOK> m;
  m.read(G, t0, wave, lane);
  float h0[4];
  auto load_dfinal = [&](int i, float (&k)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) k[e] = 0.f;
    if (a.dfin) load_state(a.dfin, GDN_F32, (int64_t)i * a.C + c, left, k);
  };
  by_marks(m, [&](auto plain) {
    constexpr bool PL = decltype(plain)::value;
    float A[4], F[4], B[4], P[4] = {1.f, 1.f, 1.f, 1.f};
    forward_map<Tx, PL>(a, m, x, g, c, left, A, F, h0);
    // the map of the carry: over all tokens, or up to the first sequence end
    int hi = PL ? TOK : m.hi;
#pragma unroll
    for (int e = 0; e < 4; ++e) B[e] = 0.f;
    if (!PL && m.last) {
      hi = __builtin_ctz(m.last) + 1;
      load_dfinal(m.seq_last(hi - 1), B);
    }
    descend<TOK>(PL ? 0 : m.lo, hi, [&](int s) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float gg = g[s][e];
        B[e] = gg * (to_f32((Tx)dy[s][e]) + B[e]);
        P[e] *= gg;
      }
    });
    if (PL) keep_above_zero<TOK>(g, P);
    *reinterpret_cast<f32x4v *>(&sA[wave][4 * lane]) = f32x4v{P[0], P[1], P[2], P[3]};
    *reinterpret_cast<f32x4v *>(&sF[wave][4 * lane]) = f32x4v{F[0], F[1], F[2], F[3]};
    *reinterpret_cast<f32x4v *>(&sB[wave][4 * lane]) = f32x4v{B[0], B[1], B[2], B[3]};
  });
  __syncthreads();

  const unsigned firsts = marked_waves(G.first, lane), lasts = marked_waves(G.last, lane);
  if (tid < kRecChannels) {
    const int ch = cb * kRecChannels + tid;
    if (ch < a.C) {
      float A = 1.f, B = 0.f, k = 0.f;
#pragma unroll
      for (int w = kWaves - 1; w >= 0; --w) {
        B = lasts >> w & 1 ? sB[w][tid] : fmaf(sA[w][tid], B, sB[w][tid]);
        A *= sA[w][tid];
      }
      if (rare(A == 0.f) && A == 0.f && all_above_zero(sA, tid)) A = kTiny;
      if (a.ticket) {
        k = chain(a, tile, ch, 1, Map{A, B, lasts != 0});
        reread_lds();
      }
      float h = a.chunk && t0 < T ? a.chunk[(int64_t)tile * a.C + ch] : 0.f;
#pragma unroll
      for (int w = kWaves - 1; w >= 0; --w) {
        const float b = sB[w][tid];
        sB[w][tid] = k;
        k = lasts >> w & 1 ? b : fmaf(sA[w][tid], k, b);
      }
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = sF[w][tid];
        sF[w][tid] = h;
        h = firsts >> w & 1 ? f : fmaf(sA[w][tid], h, f);
      }
    }
  }
  __syncthreads();

  // the last of a head's lanes writes its gate's gradient
  const bool writes_head = PH && (lane & (a.D / 4 - 1)) == a.D / 4 - 1;
  // gradients of rows outside every sequence are zero
  if (m.lo > 0 || m.hi < TOK) {
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < TOK; ++s) {
      const int64_t t = tw + s;
      if ((s < m.lo || s >= m.hi) && t < a.T && left > 0) {
        store4<Tx, VEC>((Tx *)a.dx + t * a.C + c, left, zero);
        if constexpr (PH) {
          if (writes_head) ((Tg *)a.dg)[t * a.H + head] = from_f32<Tg>(0.f);
        } else {
          store4<Tg, VEC>((Tg *)a.dg + t * a.C + c, left, zero);
        }
      }
    }
  }
  if (left > 0) {
    // Half of the wave's tokens at a time, the later half first: the states
    // before its tokens are formed again from the wave's start (half as many
    // registers as for all of them), then the gradients backward.
    float k[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) k[e] = sB[wave][4 * lane + e];
    by_marks(m, [&](auto plain) {
      constexpr bool PL = decltype(plain)::value;
#pragma unroll
      for (int half = 1; half >= 0; --half) {
        constexpr int kHalf = TOK / 2;
        const int s0 = half * kHalf, s1 = s0 + kHalf;
        float before[kHalf][4], h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = opaque(sF[wave][4 * lane + e]);
        segments_up<PL>(m, [&](int lo, int hi, bool started) {
          if (lo >= s1) return;
          if (!PL && started) start_state(a, m, lo, c, left, h0, h);
          ascend<TOK>(lo, hi, [&](int s) {
            if (s >= s1) return;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (s >= s0) before[s - s0][e] = h[e];
              h[e] = fmaf(g[s][e], h[e], to_f32((Tx)x[s][e]));
            }
          });
        });
        segments_down<PL>(m, [&](int lo, int hi, bool started) {
          if (lo >= s1 || hi <= s0) return;
          if (!PL && hi <= s1 && (m.last >> (hi - 1) & 1)) load_dfinal(m.seq_last(hi - 1), k);
          descend<TOK>(lo, hi, [&](int s) {
            if (s < s0 || s >= s1) return;
            const int64_t t = tw + s;
            float dh[4], dg[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              dh[e] = to_f32((Tx)dy[s][e]) + k[e];
              dg[e] = dh[e] * before[s - s0][e];
              k[e] = g[s][e] * dh[e];
            }
            if constexpr (PH) {
              const float sum = head_sum((dg[0] + dg[1]) + (dg[2] + dg[3]), a.D);
              if (writes_head) ((Tg *)a.dg)[t * a.H + head] = from_f32<Tg>(sum);
            } else {
              store4<Tg, VEC>((Tg *)a.dg + t * a.C + c, left, dg);
            }
            store4<Tx, VEC>((Tx *)a.dx + t * a.C + c, left, dh);
          });
          if (!PL && lo >= s0 && a.dinit && started)
            store_state(a.dinit, GDN_F32, (int64_t)m.seq_first(lo) * a.C + c, left, k);
        });
      }
    });
  }
}

// ------------------------------------------------------------------- decode

// One thread per four channels of one sequence: the state row is read,
// updated and written back.  Bounded by launch latency below a few hundred
// sequences (6 x 2048 channels: 3.0 us), by memory above (256 x 4096 channels
// with fp32 states, 17 MB: 4.4 to 5 us).
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
  const V4<Tx> x = load4<Tx, VEC>((const Tx *)a.x + i * a.x_stride + c, left);
  Gate<Tg, PH, VEC> g;
  g.load((const Tg *)a.g + i * a.g_stride, c, left, PH ? c / a.D : 0);
  float h[4];
  load_init(a, i, c, left, h);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = fmaf(g[e], h[e], to_f32((Tx)x[e]));
  store4<Tx, VEC>((Tx *)a.out + (int64_t)i * a.C + c, left, h);
  if (a.fin) store_final(a, i, c, left, h);
}

// ------------------------------------------------------------------ prepare

constexpr int kPrepThreads = 1024;

// Chain words to kPending and the tickets to zero; block 0 of a large batch
// also forms the sanitised sequence starts (running maximum of cu_seqlens
// clamped to [0, T]) and the status word.
__global__ void __launch_bounds__(kPrepThreads) rec_prepare_kernel(RecArgs a, int32_t *bos) {
  const int tid = threadIdx.x;
  if (a.ticket) {
    // tile and group words lie behind each other; 16 bytes a step (the last
    // one may be half)
    const int64_t n = ((int64_t)a.ntiles + groups_of(a.ntiles)) * a.C;
    const int64_t at = (int64_t)blockIdx.x * kPrepThreads + tid;
    const int64_t step = (int64_t)gridDim.x * kPrepThreads;
    const u32x4 ones = {~0u, ~0u, ~0u, ~0u};
    for (int64_t i = at; i < n / 2; i += step) reinterpret_cast<u32x4 *>(a.words)[i] = ones;
    if (at == 0 && n % 2) a.words[n - 1] = ~0ull;
    for (int64_t i = at; i < a.ncb; i += step) a.ticket[i * kTicketStep] = 0u;
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

// A scan's tiles, then the workgroups for empty sequences.
unsigned scan_grid(const RecArgs &a) { return a.units + (unsigned)(a.empties * a.ncb); }

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
  const int64_t n = a.ticket ? ((int64_t)a.ntiles + groups_of(a.ntiles)) * a.C : 1;
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
