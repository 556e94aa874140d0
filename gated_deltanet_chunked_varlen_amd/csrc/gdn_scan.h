// gdn_scan.h -- device-side building blocks of the selective state space scan,
// shared by its forward and its backward kernels.
#pragma once

#include "gdn_layers.h"

// Products and sums are contracted only where fmaf says so.
#pragma clang fp contract(off)

namespace gdn {
namespace scan {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRun = 8;  // tokens of which raw values are under way
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kTiny = 0x1p-149f;
constexpr float kLargest = 0x1.fffffep127f;

// Waves per SIMD that the register budget is made for.
constexpr int scan_waves(int ns) { return ns == 8 ? 4 : ns == 16 ? 3 : ns == 32 ? 2 : 1; }

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Values that are the same for the whole wave, by scalar loads.
template <typename V> __device__ __forceinline__ V uniform_load(const float *p) {
  return *(const __attribute__((address_space(4))) V *)(uintptr_t)p;
}

// log(1 + e^v) to full precision: with w = 1 + e^-|v| as rounded, log(w) carries
// the rounding of w, which the quotient takes out again.
__device__ __forceinline__ float softplus(float v) {
  const float e = __builtin_amdgcn_exp2f(-kLog2E * fabsf(v));
  const float w = 1.f + e, m = w - 1.f;
  float l = kLn2 * __builtin_amdgcn_logf(w);
  l = m == 0.f ? e : l * e * __builtin_amdgcn_rcpf(m);
  return fmaxf(v, 0.f) + (v != v ? v : l);
}

__device__ __forceinline__ float step_size(const ScanArgs &a, float v) {
  return a.softplus ? softplus(v) : v;
}

// ----------------------------------------------------------------- geometry

struct TileGeo {
  unsigned long long first[4], last[4], valid[4];
  int seq[256];
  int mark[kWaves][64];
};

__device__ __forceinline__ void tile_geometry(const ScanArgs &a, int t0, TileGeo &G) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int from = t0 & ~63, blocks = (t0 + a.L - from + 63) / 64;
  if (wave < blocks) {
    const Block64 g = block_geometry(a.b, from + 64 * wave, lane, G.mark[wave]);
    G.seq[64 * wave + lane] = g.seq;
    if (lane == 0) {
      G.first[wave] = g.first;
      G.last[wave] = g.last;
      G.valid[wave] = g.valid;
    }
  }
  __syncthreads();
}

// `n` <= 32 bits of a mask from token t of the geometry's blocks on (they do not
// cross a block).
__device__ __forceinline__ unsigned bits_at(const unsigned long long *m, int at, int n) {
  const unsigned long long w = m[at >> 6] >> (at & 63);
  return __builtin_amdgcn_readfirstlane((unsigned)w) & (n == 32 ? ~0u : (1u << n) - 1);
}

// The marks of a run of n tokens: bit i, token i.
struct Marks {
  unsigned first, last, valid;
  const int *seq;
  __device__ __forceinline__ Marks(const TileGeo &G, int at, int n)
      : first(bits_at(G.first, at, n)), last(bits_at(G.last, at, n)),
        valid(bits_at(G.valid, at, n)), seq(G.seq + at) {}
  __device__ __forceinline__ int seq_at(int i) const {
    return __builtin_amdgcn_readfirstlane(seq[i]);
  }
};

// A wave's channel: group, and channel number (ok: there is one).
struct Channel {
  int g, c;
  bool ok;
  __device__ __forceinline__ Channel(const ScanArgs &a, int cb, int lane) {
    const int per = a.ncb / a.G;  // blocks of a group
    g = cb / per;
    const int p = (cb - g * per) * 64 + lane;
    ok = p < a.P;
    c = g * a.P + (ok ? p : a.P - 1);  // others look at the group's last channel
  }
};

// One token's step of all states of a lane's channel; with OUT the sum of
// C h is added to y.  Not FULL: the states from N on, whose coefficients are 0, are
// kept at 0 also under an infinite step or input, as they are part of that sum (4096
// tokens of 4096 channels with 24 states: 353 us, 346 if they are not).
template <int NS, bool OUT, bool FULL = true>
__device__ __forceinline__ void token_step(const float *bc, float dt, float u,
                                           const float (&A2)[NS], float (&h)[NS], float &y,
                                           int N = NS) {
  constexpr int Q = NS < 16 ? NS : 16;
  constexpr int kSure = FULL ? NS : NS > 8 ? NS / 2 : 1;  // states that there are
  typedef float row __attribute__((ext_vector_type(Q)));
  float s[2] = {y, 0.f};
#pragma unroll
  for (int k = 0; k < NS; k += Q) {
    const row b = uniform_load<row>(bc + k);
    const row c = OUT ? uniform_load<row>(bc + NS + k) : row(0.f);
#pragma unroll
    for (int n = 0; n < Q; ++n) {
      const float e = __builtin_amdgcn_exp2f(dt * A2[k + n]);
      h[k + n] = k + n < kSure || k + n < N ? fmaf(e, h[k + n], u * b[n]) : 0.f;
      if (OUT) s[n & 1] = fmaf(c[n], h[k + n], s[n & 1]);
    }
  }
  if (OUT) y = s[0] + s[1];
}

// An address that is the same for all lanes, in scalar registers: 64-bit products
// are formed in vector registers even where their factors are the same for the
// whole wave, and a load then takes a vector address (six vector operations each).
template <typename T> __device__ __forceinline__ T *uniform(T *p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (T *)(uintptr_t)((uint64_t)hi << 32 | lo);
}

// Element of a lane in a row that starts `at` elements behind p: an address that
// is the same for all lanes and `bytes` of this one (so that a load takes one
// register for its address).
template <typename T> __device__ __forceinline__ const T *lane_of(const void *p, int64_t at,
                                                                  unsigned bytes) {
  return (const T *)(uniform((const char *)p + at * (int64_t)sizeof(T)) + bytes);
}
template <typename T> __device__ __forceinline__ T *lane_of(void *p, int64_t at, unsigned bytes) {
  return (T *)(uniform((char *)p + at * (int64_t)sizeof(T)) + bytes);
}

// Raw values of U tokens of one channel.
template <typename Tx, int U> struct Rows {
  Tx v[U];
  // Tokens t .. of rows `stride` elements apart, the last one in place of those
  // behind it.
  __device__ __forceinline__ void load(const void *p, int64_t stride, int t, int end, int c) {
    const int64_t step = stride * (int64_t)sizeof(Tx);
    const char *row = uniform((const char *)p + min(t, end) * step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = *(const Tx *)(row + (unsigned)c * (unsigned)sizeof(Tx));
      row += t + u < end ? step : 0;
    }
  }
};

// D x, nothing without D (0 times infinity is no number).
__device__ __forceinline__ float skip_of(const ScanArgs &a, float D, float x) {
  return a.D ? D * x : 0.f;
}

inline unsigned tile_grid(const ScanArgs &a, int empties) {
  const int rows = a.ntiles + empties;  // (without any, one for the status word)
  return (unsigned)((rows > 0 ? rows : 1) * ((a.ncb + kWaves - 1) / kWaves));
}

template <template <typename, int> class L, typename Tx>
hipError_t by_states(const ScanArgs &a, hipStream_t s) {
  switch (scan_states(a.N)) {
    case 8: return L<Tx, 8>::go(a, s);
    case 16: return L<Tx, 16>::go(a, s);
    case 32: return L<Tx, 32>::go(a, s);
    default: return L<Tx, 64>::go(a, s);
  }
}
template <template <typename, int> class L>
hipError_t dispatch(const ScanArgs &a, hipStream_t s) {
  if (a.x_dtype == GDN_F32) return by_states<L, float>(a, s);
  return a.x_dtype == GDN_BF16 ? by_states<L, bf16>(a, s) : by_states<L, f16>(a, s);
}

}  // namespace scan
}  // namespace gdn
