// k12_scan_walk.hip -- forward pass of the selective state space scan for wide
// layers: one pass along the tokens.
//
// The passes over tiles (k9_scan.hip) form every exponential twice.  Where a layer
// has enough channels to fill the GPU, a workgroup takes 16 channels and walks
// along the tokens instead, kWaves runs of TW tokens at a time, one run a wave:
//   1. every wave: its run's decays exp(d A), kept in registers, and its last
//      state from zero; both, the decay over the run and the state, into LDS
//   2. (barrier) every wave composes the states behind the waves before it, from
//      where the last step ended
//   3. every wave: the true states, from the decays it kept, and the outputs
// so that a token takes one exponential per state, and no second kernel.  A lane
// holds S states of a channel, four lanes a channel.  One prompt of 16384 tokens of
// 4096 channels with 16 states takes 487 us, the passes over tiles 803; 4096 such
// tokens 122 and 237.
//
// Bounded by the vector ALU and by what two waves per SIMD leave idle: some 45 cycles
// of a SIMD per 64 states (the exponential 8, its argument, the input's product twice,
// three fused products; the rest is the outputs' sums over four lanes and what a token
// takes for all of its states); it is busy for 74% of the time.
//
// The tokens can be cut into segments that workgroups of their own walk along:
// a segment begins with the first sequence that starts at or behind its place.
//
// A run of a wave that lies in the middle of a sequence is straight code; else its
// tokens are walked sequence by sequence.  A sequence that starts in a run and
// goes on keeps its initial state in registers for step 3: in a pool worked on in
// place another wave may have written its final state over it by then.
#include "gdn_scan.h"

#include <type_traits>

#pragma clang fp contract(off)

namespace gdn {

using namespace scan;

namespace {

constexpr int kLanes = 4;      // of a channel
constexpr int kChannels = 16;  // of a workgroup
// Tokens of which the coefficients are read together, those of the next ones while
// these are worked on: 16384 x 4096 in bf16 took 4 % longer where the compiler ordered
// the reads of four tokens.  All of a run's at once would take the registers that the
// decays are in.
constexpr int kStates = 4, kOutputs = 2;  // of the first sweep, of the second
constexpr int kCompose = 4;  // waves' states read from LDS together
constexpr int kLoadsDone = 0x0F70;  // s_waitcnt vmcnt(0), nothing else

// Tokens of a run and waves of a workgroup by the states of a lane: S TW decays
// are held in registers (16 tokens of 8 states do not fit: 4096 tokens of 4096 channels
// with 32 states took 11 % longer than with 8, 233 us), and the waves' states in LDS.
constexpr int run_tokens(int s) { return s <= 4 ? 16 : 8; }
constexpr int run_waves(int s) { return s <= 8 ? 8 : 4; }

template <int CTRL> __device__ __forceinline__ float quad(float x) {
  return __uint_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xF, 0xF, true));
}
// Element of a lane, `bytes` behind an element that is the same for all lanes (whose
// address is left to vector registers: scalar ones are short here).
template <typename T> __device__ __forceinline__ T *shared_row(const void *p, int64_t at,
                                                               unsigned bytes) {
  return (T *)((char *)const_cast<void *>(p) + at * (int64_t)sizeof(T) + bytes);
}
// The value that lane k of each quad holds.
__device__ __forceinline__ float quad_lane(float x, int k) {
  return k == 0 ? quad<0x00>(x) : k == 1 ? quad<0x55>(x) : k == 2 ? quad<0xAA>(x) : quad<0xFF>(x);
}
__device__ __forceinline__ float quad_sum(float x) {
  x += quad<0xB1>(x);
  return x + quad<0x4E>(x);
}

// First token at or behind t0 where a sequence may start (a cut between two).
__device__ __forceinline__ int cut_at(const Batch &b, const SeqLane &s, int t0, int lane) {
  if (!b.bos) {
    int v = lane <= b.N && s.bos >= t0 ? s.bos : (int)b.T;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = min(v, __shfl_xor(v, o));
    return __builtin_amdgcn_readfirstlane(v);
  }
  int lo = 0, hi = b.N;  // the first bos[i] >= t0, at most bos[N]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (b.bos[mid] >= t0) hi = mid;
    else lo = mid + 1;
  }
  const int at = b.bos[lo];
  return at >= t0 ? min(at, (int)b.T) : (int)b.T;
}

template <typename Tx, int S>
__global__ void __launch_bounds__(64 * run_waves(S), S <= 8 ? 2 : 1)
    scan_walk_kernel(ScanArgs a) {
  constexpr int TW = run_tokens(S), WAVES = run_waves(S), NS = kLanes * S, TQ = TW / kLanes;
  constexpr int NV = TW * 2 * NS / 8 / 64 > 0 ? TW * 2 * NS / 8 / 64 : 1;  // vectors of B and C
  constexpr unsigned kAll = (1u << TW) - 1;
  __shared__ float s_bc[WAVES][TW][2][NS];
  __shared__ Vec<float, S> s_state[2][WAVES][64], s_decay[2][WAVES][64], s_carry[2][64];
  __shared__ int s_reset[2][WAVES];
  __shared__ int s_mark[WAVES][64], s_seq[WAVES][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane & 3;
  if (blockIdx.x == 0 && wave == 0 && a.b.status && !a.b.bos) batch_status(a.b, lane);
  // neighbouring blocks of channels share cache lines: eight sets of neighbours,
  // as workgroups go to the eight XCDs in turn
  const int per = (a.ncb + 7) / 8, set = 8 * per;
  const int seg = blockIdx.x / set, at = blockIdx.x % set;
  const int cb = (at & 7) * per + (at >> 3);
  if (seg >= a.nseg) {  // the workgroups behind: empty sequences
    constexpr int U = 4;
    const int64_t row = (int64_t)a.C * a.N, step = (int64_t)set * blockDim.x;
    for (int i = seg - a.nseg; i < a.b.N; i += a.empties) {
      int bos, len;
      sequence_of(a.b, i, lane, bos, len);
      const int64_t r = state_row(a.b, i);
      if (len != 0 || r < 0) continue;
      for (int64_t e = (int64_t)at * blockDim.x + threadIdx.x; e < row; e += U * step) {
        int64_t from[U], to[U];
        float v[U][1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t k = min(e + u * step, row - 1);
          from[u] = r * a.init.stride + k;
          to[u] = r * a.fin.stride + k;
          v[u][0] = 0.f;
        }
        if (a.init.p) state_read<U, 1>(a.init, from, v);
        state_write<U, 1>(a.fin, to, v);
      }
    }
    return;
  }
  if (cb >= a.ncb) return;
  const int blocks = a.ncb / a.G, g = cb / blocks;
  const int p = (cb - g * blocks) * kChannels + (lane >> 2);
  const bool ok = p < a.P;
  const int c = g * a.P + (ok ? p : a.P - 1);
  SeqLane seqs{};
  if (!a.b.bos) seqs = seq_lane(a.b.cu, a.b.cu_type, a.b.N, a.b.T, lane);
  const int T = (int)a.b.T, share = (T + a.nseg - 1) / a.nseg, end = T - 1;
  const int from = seg == 0 ? 0 : cut_at(a.b, seqs, seg * share, lane);
  const int to = seg == a.nseg - 1 ? T : cut_at(a.b, seqs, (seg + 1) * share, lane);
  if (from >= to) return;

  float A2[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    A2[s] = kLog2E * a.A[(int64_t)c * NS + q * S + s];
  }
  const float bias = a.dbias ? a.dbias[c] : 0.f, D = a.D ? a.D[c] : 0.f;

  // this lane's states of sequence i, before its first token and behind its last
  auto initial = [&](int i, float(&h)[S]) {
#pragma unroll
    for (int s = 0; s < S; ++s) h[s] = 0.f;
    const int64_t r = a.init.p ? state_row(a.b, i) : -1;
    if (r < 0) return;
    const Vec<float, S> v = load_vec<float, S>(
        shared_row<float>(a.init.p, r * a.init.stride, (unsigned)(c * NS + q * S) * 4));
#pragma unroll
    for (int s = 0; s < S; ++s) h[s] = v.e[s];
  };
  auto final = [&](int i, const float(&h)[S]) {
    const int64_t r = state_row(a.b, i);
    if (r < 0 || !ok) return;
    store_vec<float, S>(
        shared_row<float>(a.fin.p, r * a.fin.stride, (unsigned)(c * NS + q * S) * 4), h);
  };

  // raw values of the next run: lane q of a channel holds tokens q TQ .. of it
  // (without z, x in its place: a load less under a condition)
  Tx rx[TQ], rd[TQ], rz[TQ];
  Vec<Tx, 8> rbc[NV];
  const Tx *const zsrc = (const Tx *)(a.z ? a.z : a.x);
  const int64_t zstep = a.z ? a.z_stride : a.x_stride;
  constexpr int kStep = WAVES * TW;
  const int base0 = from / kStep * kStep;
  // this lane's first token of the run that is fetched next, and of the one written
  const int64_t t00 = base0 + wave * TW + q * TQ;
  const Tx *xp = (const Tx *)a.x + t00 * a.x_stride + c;
  const Tx *dp = (const Tx *)a.delta + t00 * a.delta_stride + c;
  const Tx *zp = zsrc + t00 * zstep + c;
  Tx *op = (Tx *)a.out + (t00 - kStep) * a.C + c;  // (of the run before)
  auto fetch = [&](int t0) {
    if (t0 + TW <= T) {
      const Tx *x = xp, *d = dp, *z = zp;
#pragma unroll
      for (int k = 0; k < TQ; ++k, x += a.x_stride, d += a.delta_stride, z += zstep) {
        rx[k] = *x;
        rd[k] = *d;
        rz[k] = *z;
      }
    } else {
#pragma unroll
      for (int k = 0; k < TQ; ++k) {
        const int64_t t = min(t0 + q * TQ + k, end);
        rx[k] = ((const Tx *)a.x)[t * a.x_stride + c];
        rd[k] = ((const Tx *)a.delta)[t * a.delta_stride + c];
        rz[k] = zsrc[t * zstep + c];
      }
    }
    xp += kStep * a.x_stride;
    dp += kStep * a.delta_stride;
    zp += kStep * zstep;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int id = v * 64 + lane, n0 = id % (NS / 8) * 8, which = id / (NS / 8) % 2;
      const int64_t t = min(t0 + min(id / (2 * NS / 8), TW - 1), end);
      const Tx *row = (which ? (const Tx *)a.C_ + t * a.c_stride : (const Tx *)a.B + t * a.b_stride) +
                      (int64_t)g * a.N;
      rbc[v] = load_vec<Tx, 8>(row + n0);
    }
  };

  // The outputs of a run are stored behind the waits of the next one, before its
  // fetch: stores and loads end in order, and the values that were fetched would
  // else be waited for until the stores behind them are done.
  Tx out[TQ];
  unsigned outs = 0;
  auto put = [&]() {
#pragma unroll
    for (int k = 0; k < TQ; ++k)
      if (outs >> k & 1) op[k * (int64_t)a.C] = out[k];
    op += (int64_t)kStep * a.C;
  };
  int turn = 0, within = 0, until = 0;
  int base = base0;
  fetch(base + wave * TW);
  if (wave == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) s_carry[0][lane].e[s] = 0.f;
  }
  for (; base < to; base += kStep, turn ^= 1) {
    const int t0 = base + wave * TW;
    // marks of the run; in the middle of the sequence that the last one ended in
    // there are none to look for
    unsigned valid = kAll, first = 0, last = 0;
    if (!(t0 > within && t0 + TW < until)) {
      const int b0 = t0 & ~63, sh = t0 & 63;
      const Block64 m = block_geometry(a.b, b0, lane, s_mark[wave], a.b.bos ? nullptr : &seqs);
      s_seq[wave][lane] = m.seq;
      wave_sync();
      valid = (unsigned)(m.valid >> sh) & kAll;
      first = (unsigned)(m.first >> sh) & kAll;
      last = (unsigned)(m.last >> sh) & kAll;
      // of this segment
      const int lo = max(from - t0, 0), hi = min(to - t0, TW);
      const unsigned in = lo >= TW || hi <= lo ? 0u : (kAll >> (TW - (hi - lo))) << lo;
      valid &= in;
      first &= in;
      last &= in;
      // the sequence of the run's last token, as far as this segment goes
      const int i = __builtin_amdgcn_readlane(m.seq, min(sh + TW - 1, 63));
      within = until = 0;
      if (i >= 0) {
        int bos, len;
        sequence_of(a.b, i, lane, bos, len, a.b.bos ? nullptr : &seqs);
        within = max(bos, from);
        until = min(bos + len, to);
      }
    }
    const int *seq = s_seq[wave] + (t0 & 63);
    auto seq_at = [&](int t) { return __builtin_amdgcn_readfirstlane(seq[t]); };
    float dt[TQ], u[TQ];
    Tx x[TQ], z[TQ];
#pragma unroll
    for (int k = 0; k < TQ; ++k) {
      const bool in = valid >> (q * TQ + k) & 1;
      x[k] = rx[k];
      z[k] = rz[k];
      dt[k] = in ? step_size(a, to_f32(rd[k]) + bias) : 0.f;
      u[k] = in ? dt[k] * to_f32(rx[k]) : 0.f;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int id = v * 64 + lane;
      float f[8];
      widen(rbc[v], f);
      if (id < TW * 2 * NS / 8) {
        f32x4 *o = (f32x4 *)(&s_bc[wave][0][0][0] + id * 8);
        o[0] = f32x4{f[0], f[1], f[2], f[3]};
        o[1] = f32x4{f[4], f[5], f[6], f[7]};
      }
    }
    wave_sync();
    put();
    if (base + kStep < to) fetch(t0 + kStep);
    auto coeff = [&](int t, int which, float(&o)[S]) {
#pragma unroll
      for (int s = 0; s < S; s += S < 4 ? S : 4) {
        const auto v = *reinterpret_cast<const Vec<float, (S < 4 ? S : 4)> *>(
            &s_bc[wave][t][which][q * S + s]);
#pragma unroll
        for (int k = 0; k < (S < 4 ? S : 4); ++k) o[s + k] = v.e[k];
      }
    };

    // f(lo, hi, whether token lo starts a sequence) for the sequences' parts of
    // the run, one after the other
    auto parts = [&](auto f) {
      unsigned left = first;
      int lo = valid ? __builtin_ctz(valid) : TW;
      bool starts = first >> (lo & 31) & 1 && lo < TW;
      const int stop = valid ? 32 - __builtin_clz(valid) : 0;
      while (lo < stop) {
        if (starts) left &= left - 1;
        const int hi = left ? __builtin_ctz(left) : stop;
        f(lo, hi, starts);
        lo = hi;
        starts = true;
      }
    };
    const bool plain = valid == kAll && (first | last) == 0;

    // 1. decays, the run's last state from zero
    float e[TW][S], h[S], h0[S];
#pragma unroll
    for (int s = 0; s < S; ++s) h[s] = h0[s] = 0.f;
    auto step1 = [&](int t, const float(&b)[S]) {
      const float d = quad_lane(dt[t % TQ], t / TQ), v = quad_lane(u[t % TQ], t / TQ);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        e[t][s] = __builtin_amdgcn_exp2f(d * A2[s]);
        h[s] = fmaf(e[t][s], h[s], v * b[s]);
      }
    };
    auto sweep1 = [&](int lo, int hi, auto all) {
      constexpr bool ALL = decltype(all)::value;
      if constexpr (ALL) {
        constexpr int K = kStates;
        float b[2][K][S];
#pragma unroll
        for (int k = 0; k < K; ++k) coeff(k, 0, b[0][k]);
#pragma unroll
        for (int t = 0; t < TW; t += K) {
          if (t + K < TW) {
#pragma unroll
            for (int k = 0; k < K; ++k) coeff(t + K + k, 0, b[(t / K + 1) & 1][k]);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int k = 0; k < K; ++k) step1(t + k, b[(t / K) & 1][k]);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int t = 0; t < TW; ++t) {
          if (t < lo || t >= hi) continue;
          float b[S];
          coeff(t, 0, b);
          step1(t, b);
        }
      }
    };
    if (plain) {
      sweep1(0, TW, std::true_type{});
    } else {
#pragma unroll
      for (int t = 0; t < TW; ++t)
#pragma unroll
        for (int s = 0; s < S; ++s) e[t][s] = 1.f;
      parts([&](int lo, int hi, bool starts) {
        if (starts) {
          initial(seq_at(lo), h0);
#pragma unroll
          for (int s = 0; s < S; ++s) h[s] = h0[s];
        }
        sweep1(lo, hi, std::false_type{});
      });
      // the states read here are there; else the other branch would wait for them
      // too, and with them for the next run's values
      __builtin_amdgcn_s_waitcnt(kLoadsDone);
    }
    float span = 0.f;
#pragma unroll
    for (int k = 0; k < TQ; ++k) span += dt[k];
    span = quad_sum(span);
    {
      Vec<float, S> hs, es;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        hs.e[s] = h[s];
        // (neither 0 nor infinite: 0 times infinity is no number)
        es.e[s] = __builtin_amdgcn_fmed3f(__builtin_amdgcn_exp2f(span * A2[s]), kTiny, kLargest);
      }
      s_state[turn][wave][lane] = hs;
      s_decay[turn][wave][lane] = es;
    }
    if (lane == 0) s_reset[turn][wave] = first != 0;
    __syncthreads();

    // 2. the state before the run
    float cr[S];
#pragma unroll
    for (int s = 0; s < S; ++s) cr[s] = s_carry[turn][lane].e[s];
    const unsigned resets = (unsigned)__ballot(s_reset[turn][lane % WAVES] != 0);
#pragma unroll
    for (int j0 = 0; j0 < WAVES - 1; j0 += kCompose) {
      if (j0 >= wave) break;
      Vec<float, S> hj[kCompose], ej[kCompose];
#pragma unroll
      for (int j = 0; j < kCompose; ++j) {
        hj[j] = s_state[turn][min(j0 + j, WAVES - 1)][lane];
        ej[j] = s_decay[turn][min(j0 + j, WAVES - 1)][lane];
      }
#pragma unroll
      for (int j = 0; j < kCompose; ++j) {
        if (j0 + j >= wave) continue;
        const bool reset = resets >> (j0 + j) & 1;
#pragma unroll
        for (int s = 0; s < S; ++s)
          cr[s] = reset ? hj[j].e[s] : fmaf(ej[j].e[s], cr[s], hj[j].e[s]);
      }
    }
    // (0 where no earlier token of this segment is a sequence's)
    if (a.chunk && t0 % a.L == 0 && t0 >= from && t0 < to && ok) {
      float *row = a.chunk + (int64_t)(t0 / a.L) * NS * a.C + c;
#pragma unroll
      for (int s = 0; s < S; ++s) row[(int64_t)(q * S + s) * a.C] = cr[s];
    }

    // 3. the true states and the outputs
    float y[TQ];
#pragma unroll
    for (int k = 0; k < TQ; ++k) y[k] = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) h[s] = cr[s];
    auto step2 = [&](int t, const float(&b)[S], const float(&cc)[S]) {
      const float v = quad_lane(u[t % TQ], t / TQ);
      float o = 0.f;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        h[s] = fmaf(e[t][s], h[s], v * b[s]);
        o = fmaf(cc[s], h[s], o);
      }
      o = quad_sum(o);
      y[t % TQ] = q == t / TQ ? o : y[t % TQ];
    };
    auto sweep2 = [&](int lo, int hi, auto all) {
      constexpr bool ALL = decltype(all)::value;
      if constexpr (ALL) {
        constexpr int K = kOutputs;
        float b[2][K][S], cc[2][K][S];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          coeff(k, 0, b[0][k]);
          coeff(k, 1, cc[0][k]);
        }
#pragma unroll
        for (int t = 0; t < TW; t += K) {
          if (t + K < TW) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
              coeff(t + K + k, 0, b[(t / K + 1) & 1][k]);
              coeff(t + K + k, 1, cc[(t / K + 1) & 1][k]);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int k = 0; k < K; ++k) step2(t + k, b[(t / K) & 1][k], cc[(t / K) & 1][k]);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int t = 0; t < TW; ++t) {
          if (t < lo || t >= hi) continue;
          float b[S], cc[S];
          coeff(t, 0, b);
          coeff(t, 1, cc);
          step2(t, b, cc);
        }
      }
    };
    if (plain) {
      sweep2(0, TW, std::true_type{});
    } else {
      parts([&](int lo, int hi, bool starts) {
        if (starts) {
          if (first >> lo == 1u) {  // the last start: another wave may have its end
#pragma unroll
            for (int s = 0; s < S; ++s) h[s] = h0[s];
          } else {
            initial(seq_at(lo), h);
          }
        }
        sweep2(lo, hi, std::false_type{});
        if (a.fin.p && (last >> (hi - 1) & 1)) final(seq_at(hi - 1), h);
      });
      __builtin_amdgcn_s_waitcnt(kLoadsDone);
    }
    if (wave == WAVES - 1) {
#pragma unroll
      for (int s = 0; s < S; ++s) s_carry[turn ^ 1][lane].e[s] = h[s];
    }
#pragma unroll
    for (int k = 0; k < TQ; ++k) {
      float o = a.D ? fmaf(D, to_f32(x[k]), y[k]) : y[k];
      if (a.z) {
        const float zz = to_f32(z[k]);
        o *= zz * sigmoid(zz);
      }
      out[k] = from_f32<Tx>(o);
    }
    outs = ok ? valid >> q * TQ : 0u;
  }
  put();
}

template <typename Tx, int NS> struct Walk {
  static hipError_t go(const ScanArgs &a, hipStream_t s) {
    constexpr int S = NS / kLanes;
    const unsigned set = 8u * (unsigned)((a.ncb + 7) / 8);
    scan_walk_kernel<Tx, S><<<dim3(set * (unsigned)(a.nseg + a.empties)),
                              dim3(64 * run_waves(S)), 0, s>>>(a);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_scan_walk(const ScanArgs &a, hipStream_t s) { return dispatch<Walk>(a, s); }

}  // namespace gdn
