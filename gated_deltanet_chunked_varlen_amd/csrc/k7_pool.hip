// k7_pool.hip -- rows of a state pool: copied (forked, moved, brought in from
// another pool or type), zeroed, compacted.
//
// A row of a gated-delta pool is H x V x K elements (1 MB at 16 heads of 128 x
// 128 fp32), one of a recurrence pool H x D (8 KB at 16 x 128), so the work is
// cut into units of about kUnitBytes: a slice of one long row, or several
// short rows.  Bounded by HBM (each byte moved once each way) for long rows
// and by launch latency for a few short ones; every call is one kernel.
//
// Row lists live on the device, so who copies what is settled there: each
// workgroup reads the whole list for its own entries instead of waiting for a
// planning kernel.  That is meant for lists of up to a few thousand entries
// (4-byte words from L2, less than the rows); a copy's time grows with the
// square of its list, which is why it takes at most GDN_POOL_MAX_ROWS entries.
//
// Measured: four 1 MB rows into 32 (38 MB): 10 us, 3 of them a launch's least;
// 96 rows from bf16 to fp32 (302 MB): 66 us, 4.6 TB/s; 64 rows of 1 MB zeroed:
// 11.8 us, 5.7 TB/s; 64 rows of 512 KB moved by a compaction (67 MB): 15 us;
// one row of 1 MB from bf16 to 2 MB of fp32: 5.9 us a call.
// Units of 32 and 128 KB and two to four times the loads in flight were no
// faster (38 MB fork: 10.6 and 16.2 us with 32 and 128 KB units).
#include "gdn_common.h"
#include "gdn_internal.h"
#include "gdn_recurrence.h"

#include <type_traits>

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kUnitBytes = 64 << 10;
constexpr int kMaxGroup = 16;  // short rows per unit
constexpr int kBatch = 4;      // loads in flight per thread

// Row numbers: the list entry, -1 for padding, -2 for entries outside the pool.
__device__ __forceinline__ int list_row(const void *list, int type, int64_t i, int64_t pool) {
  const int64_t r = load_index_any(list, type, i);
  return r == -1 ? -1 : (r < 0 || r >= pool) ? -2 : (int)r;
}

// ------------------------------------------------------------ moving elements

__device__ __forceinline__ int64_t row_offset(const int64_t *str, int64_t d2, int64_t d3,
                                              int64_t e) {
  const int64_t k = e % d3, r = e / d3;
  return (r / d2) * str[1] + (r % d2) * str[2] + k * str[3];
}

__host__ __device__ constexpr int elem_size(int dtype) {
  return dtype == GDN_F32 ? 4 : dtype == GDN_BF16 || dtype == GDN_F16 ? 2 : 1;
}

__device__ __forceinline__ const char *src_row(const PoolArgs &a, int r) {
  return (const char *)a.src + (int64_t)r * a.src_str[0] * elem_size(a.src_dtype);
}
__device__ __forceinline__ char *dst_row(const PoolArgs &a, int r) {
  return (char *)a.dst + (int64_t)r * a.dst_str[0] * elem_size(a.dst_dtype);
}

// Bytes b0 .. b1 - 1 of a contiguous row by the whole workgroup, in vectors V:
// copied, or (ZERO) cleared.  kBatch loads per thread are on their way before
// the first store; `go` is asked in between, so that whatever decides whether
// the row is written runs beside them.
template <typename V, bool ZERO, typename F>
__device__ __forceinline__ void move_bytes(const char *src, char *dst, int64_t b0, int64_t b1,
                                           F go) {
  constexpr int64_t step = sizeof(V) * kThreads;
  int64_t b = b0 + (int64_t)sizeof(V) * threadIdx.x;
  if constexpr (ZERO) {
    if (!go()) return;
#pragma unroll 4
    for (; b < b1; b += step) *(V *)(dst + b) = V{};
    return;
  }
  V v[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i)
    if (b + i * step < b1) v[i] = *(const V *)(src + b + i * step);
  if (!go()) return;
  for (;;) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (b + i * step < b1) *(V *)(dst + b + i * step) = v[i];
    b += kBatch * step;
    if (b - (int64_t)sizeof(V) * threadIdx.x >= b1) return;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (b + i * step < b1) v[i] = *(const V *)(src + b + i * step);
  }
}

template <typename U, bool ZERO>
__device__ __forceinline__ void move_strided(const PoolArgs &a, const U *src, U *dst, int64_t e0,
                                             int64_t e1) {
#pragma unroll 1
  for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads)
    dst[row_offset(a.dst_str, a.d2, a.d3, e)] =
        ZERO ? (U)0 : src[row_offset(a.src_str, a.d2, a.d3, e)];
}

// Elements e0 .. e1 - 1 of row s (ZERO: zeros) into row d of the same type, bit
// for bit.
template <bool ZERO, typename F>
__device__ __forceinline__ void move_equal(const PoolArgs &a, int s, int d, int64_t e0, int64_t e1,
                                           F go) {
  const int es = elem_size(a.dst_dtype);
  const char *src = ZERO ? nullptr : src_row(a, s);
  char *dst = dst_row(a, d);
  if (a.flat) {
    if (a.align >= 16) move_bytes<u32x4, ZERO>(src, dst, e0 * es, e1 * es, go);
    else if (es == 4) move_bytes<uint32_t, ZERO>(src, dst, e0 * es, e1 * es, go);
    else if (es == 2) move_bytes<uint16_t, ZERO>(src, dst, e0 * es, e1 * es, go);
    else move_bytes<uint8_t, ZERO>(src, dst, e0 * es, e1 * es, go);
  } else if (go()) {
    if (es == 4) move_strided<uint32_t, ZERO>(a, (const uint32_t *)src, (uint32_t *)dst, e0, e1);
    else if (es == 2)
      move_strided<uint16_t, ZERO>(a, (const uint16_t *)src, (uint16_t *)dst, e0, e1);
    else move_strided<uint8_t, ZERO>(a, (const uint8_t *)src, (uint8_t *)dst, e0, e1);
  }
}

// The same between two types, 16 bytes of the wider one per thread and step
// where every row allows it.
template <typename S, typename D, typename F>
__device__ __forceinline__ void move_convert(const PoolArgs &a, int s, int d, int64_t e0,
                                             int64_t e1, F go) {
  const S *src = (const S *)src_row(a, s);
  D *dst = (D *)dst_row(a, d);
  constexpr int W = 16 / (sizeof(S) > sizeof(D) ? sizeof(S) : sizeof(D));
  struct alignas(sizeof(S) * W) SV { S e[W]; };
  struct alignas(sizeof(D) * W) DV { D e[W]; };
  if (!a.flat || a.align < 16) {
    if (!go()) return;
#pragma unroll 1
    for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads)
      dst[row_offset(a.dst_str, a.d2, a.d3, e)] =
          from_f32<D>(to_f32(src[row_offset(a.src_str, a.d2, a.d3, e)]));
    return;
  }
  // rows are whole 16-byte groups in both types, so W divides e0 and e1
  const SV *sv = reinterpret_cast<const SV *>(src);
  DV *dv = reinterpret_cast<DV *>(dst);
  int64_t i = e0 / W + threadIdx.x;
  const int64_t end = e1 / W;
  SV v[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    if (i + j * kThreads < end) v[j] = sv[i + j * kThreads];
  if (!go()) return;
  for (;;) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      DV o;
#pragma unroll
      for (int w = 0; w < W; ++w) o.e[w] = from_f32<D>(to_f32(v[j].e[w]));
      if (i + j * kThreads < end) dv[i + j * kThreads] = o;
    }
    i += kBatch * kThreads;
    if (i - (int64_t)threadIdx.x >= end) return;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (i + j * kThreads < end) v[j] = sv[i + j * kThreads];
  }
}

// Units of a call: `group` entries by one slice of `slice` elements each.
struct Units {
  int group;
  int64_t slice;
  unsigned slices, total;  // slices of a row; units in all, below 2^31
};

Units cut(const PoolArgs &a, int64_t entries) {
  const int ss = a.src ? elem_size(a.src_dtype) : 0, ds = elem_size(a.dst_dtype);
  const int64_t es = ss > ds ? ss : ds;
  Units u;
  // slices of whole 16-byte groups in any type: multiples of 16 elements
  u.slice = kUnitBytes / es;
  if (u.slice >= a.row) {
    u.slice = a.row;
    const int64_t fit = kUnitBytes / (a.row * es);
    // no fewer units than two per compute unit for the sake of larger ones
    const int64_t spread = entries / (2 * (int64_t)a.num_cus);
    int64_t g = fit < spread ? fit : spread;
    u.group = (int)(g < 1 || !a.src ? 1 : g > kMaxGroup ? kMaxGroup : g);
  } else {
    u.group = 1;
  }
  const int64_t groups = (entries + u.group - 1) / u.group;
  auto slices = [&]() { return (a.row + u.slice - 1) / u.slice; };
  while (groups * slices() > INT32_MAX) u.slice *= 2;
  u.slices = (unsigned)slices();
  u.total = (unsigned)(groups * u.slices);
  return u;
}

unsigned unit_grid(const PoolArgs &a, const Units &u) {
  const unsigned most = 16u * (unsigned)a.num_cus;
  return u.total < most ? u.total : most;
}

// ---------------------------------------------------------------- copy, reset

// The status word of a list, by one workgroup of its own: out-of-range
// entries, destinations named twice, sources that another entry overwrites.
__device__ __forceinline__ void list_status(const PoolArgs &a, unsigned *map) {
  __shared__ unsigned s_bits;
  const int words = (int)((a.dst_pool + 31) / 32);
  for (int i = threadIdx.x; i < words; i += kThreads) map[i] = 0u;
  if (threadIdx.x == 0) s_bits = 0u;
  __syncthreads();
  unsigned bits = 0;
  for (int64_t i = threadIdx.x; i < a.count; i += kThreads) {
    const int d = list_row(a.dst_rows, a.rows_type, i, a.dst_pool);
    const int s = a.src ? list_row(a.src_rows, a.rows_type, i, a.src_pool) : 0;
    if (d == -2 || s == -2) bits |= GDN_STATUS_POOL_ROW;
    // zeroing a row twice is no conflict
    if (d >= 0 && s >= 0 && a.src && (atomicOr(&map[d >> 5], 1u << (d & 31)) >> (d & 31) & 1))
      bits |= GDN_STATUS_POOL_DUPLICATE;
  }
  __syncthreads();
  if (a.same) {
    // the rows that change: destinations of entries other than a row onto itself
    for (int i = threadIdx.x; i < words; i += kThreads) map[i] = 0u;
    __syncthreads();
    for (int pass = 0; pass < 2; ++pass) {
      for (int64_t i = threadIdx.x; i < a.count; i += kThreads) {
        const int d = list_row(a.dst_rows, a.rows_type, i, a.dst_pool);
        const int s = list_row(a.src_rows, a.rows_type, i, a.src_pool);
        if (d < 0 || s < 0 || s == d) continue;
        if (pass == 0) atomicOr(&map[d >> 5], 1u << (d & 31));
        else if (s < a.dst_pool && (map[s >> 5] >> (s & 31) & 1)) bits |= GDN_STATUS_POOL_OVERLAP;
      }
      __syncthreads();
    }
  }
  if (bits) atomicOr(&s_bits, bits);
  __syncthreads();
  if (threadIdx.x == 0) a.status[0] = (int32_t)s_bits;
}

// Entry j (source sj, destination dj) keeps entry i from acting: it has the same
// destination and comes later, or it changes entry i's source row.
__device__ __forceinline__ bool conflict(const PoolArgs &a, int64_t j, int sj, int dj, int64_t i,
                                         int si, int di) {
  return (j > i && dj == di) || (a.same && j != i && dj == si && sj != dj && si != di);
}

// Some entry of the list keeps entry i from acting; for the whole workgroup.
__device__ __forceinline__ bool skipped(const PoolArgs &a, int64_t i, int si, int di) {
  bool hit = false;
  for (int64_t j = threadIdx.x; j < a.count; j += kThreads) {
    const int d = list_row(a.dst_rows, a.rows_type, j, a.dst_pool);
    const int s = list_row(a.src_rows, a.rows_type, j, a.src_pool);
    if (d >= 0 && s >= 0) hit |= conflict(a, j, s, d, i, si, di);
  }
  return __syncthreads_or(hit) != 0;
}

// Which entries act: entry i is skipped if a later entry has its destination,
// or (in one pool) if another entry's destination is its source, unless that
// entry copies the row onto itself (such an entry has nothing to do, but wins its
// destination).  Entries with a row outside its pool take no part.
//
// MOVE::row moves elements of a row; MOVE::kZero: there are no sources.
template <typename MOVE>
__global__ void __launch_bounds__(kThreads) pool_list_kernel(PoolArgs a, Units u) {
  extern __shared__ unsigned map[];
  if (a.status && blockIdx.x == gridDim.x - 1) return list_status(a, map);
  const unsigned workers = gridDim.x - (a.status ? 1u : 0u);
  constexpr bool kZero = MOVE::kZero;
  if (kZero || u.group == 1) {
    // long rows (and zeroed ones, which have no list to check): one entry at a
    // time, its rows read as scalars
    int64_t seen = -1;
    int src = -1, dst = -1;
    for (unsigned unit = blockIdx.x; unit < u.total; unit += workers) {
      const int64_t i = unit / u.slices, e0 = unit % u.slices * u.slice;
      const int64_t e1 = e0 + u.slice < a.row ? e0 + u.slice : a.row;
      const bool fresh = i != seen;
      if (fresh) {
        seen = i;
        dst = list_row(a.dst_rows, a.rows_type, i, a.dst_pool);
        src = kZero ? 0 : list_row(a.src_rows, a.rows_type, i, a.src_pool);
      }
      if (dst < 0 || src < 0 || (!kZero && a.same && src == dst)) continue;
      if constexpr (kZero) {
        MOVE::row(a, src, dst, e0, e1, []() { return true; });
      } else {
        bool act = true;
        MOVE::row(a, src, dst, e0, e1, [&]() {
          if (fresh) act = !skipped(a, i, src, dst);
          return act;
        });
        if (!act) dst = -1;
      }
    }
    return;
  }
  __shared__ int s_src[kMaxGroup], s_dst[kMaxGroup], s_skip[kMaxGroup];
  for (unsigned unit = blockIdx.x; unit < u.total; unit += workers) {
    // short rows: a group of entries, each whole
    const int64_t i0 = (int64_t)unit * u.group;
    const int n = (int)(a.count - i0 < u.group ? a.count - i0 : u.group);
    __syncthreads();
    if ((int)threadIdx.x < n) {
      const int d = list_row(a.dst_rows, a.rows_type, i0 + threadIdx.x, a.dst_pool);
      const int s = list_row(a.src_rows, a.rows_type, i0 + threadIdx.x, a.src_pool);
      s_src[threadIdx.x] = s;
      s_dst[threadIdx.x] = d;
      s_skip[threadIdx.x] = d < 0 || s < 0 || (a.same && s == d);
    }
    __syncthreads();
    for (int64_t j = threadIdx.x; j < a.count; j += kThreads) {
      const int d = list_row(a.dst_rows, a.rows_type, j, a.dst_pool);
      const int s = list_row(a.src_rows, a.rows_type, j, a.src_pool);
      if (d < 0 || s < 0) continue;
      for (int p = 0; p < n; ++p)
        if (conflict(a, j, s, d, i0 + p, s_src[p], s_dst[p])) s_skip[p] = 1;
    }
    __syncthreads();
    for (int p = 0; p < n; ++p)
      if (!s_skip[p]) MOVE::row(a, s_src[p], s_dst[p], 0, a.row, []() { return true; });
  }
}

template <bool ZERO> struct MoveEqual {
  static constexpr bool kZero = ZERO;
  template <typename F>
  __device__ __forceinline__ static void row(const PoolArgs &a, int s, int d, int64_t e0,
                                             int64_t e1, F go) {
    move_equal<ZERO>(a, s, d, e0, e1, go);
  }
};
template <typename S, typename D> struct MoveConvert {
  static constexpr bool kZero = false;
  template <typename F>
  __device__ __forceinline__ static void row(const PoolArgs &a, int s, int d, int64_t e0,
                                             int64_t e1, F go) {
    move_convert<S, D>(a, s, d, e0, e1, go);
  }
};

// -------------------------------------------------------------------- compact

// Exclusive prefix sum over the workgroup of one value per thread; total in sh[0].
__device__ __forceinline__ int block_prefix(int x, int *sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int inc = wave_prefix_sum_i(x);
  __syncthreads();
  if (lane == 63) sh[1 + wave] = inc;
  __syncthreads();
  int pre = 0, total = 0;
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < wave) pre += sh[1 + w];
    total += sh[1 + w];
  }
  if (threadIdx.x == 0) sh[0] = total;
  __syncthreads();
  return pre + inc - x;
}

// Position of the k-th set bit of x (k < popcount).
__device__ __forceinline__ int nth_bit(unsigned x, int k) {
  for (; k > 0; --k) x &= x - 1;
  return __ffs((int)x) - 1;
}

// Every workgroup forms the plan for itself in LDS: a bitmap of the live rows
// and, per 32-row word, how many rows before it are live behind the new end
// (movers) or free before it (holes).  The k-th mover and the k-th hole then
// are two searches.  One launch, and nothing to hand over between workgroups
// (a planning launch of its own would cost more than the few microseconds that
// each workgroup spends here).
__global__ void __launch_bounds__(kThreads) pool_compact_kernel(PoolArgs a, Units u, int nwords) {
  extern __shared__ unsigned map[];  // live bits
  int *movers = (int *)(map + nwords), *holes = movers + nwords;
  __shared__ int sh[1 + kThreads / 64];
  __shared__ int s_src[kMaxGroup], s_dst[kMaxGroup];
  __shared__ unsigned s_bits;
  const int tid = threadIdx.x;
  for (int i = tid; i < nwords; i += kThreads) map[i] = 0u;
  if (tid == 0) s_bits = 0u;
  __syncthreads();
  for (int64_t i = tid; i < a.count; i += kThreads) {
    const int r = list_row(a.dst_rows, a.rows_type, i, a.dst_pool);
    if (r >= 0) atomicOr(&map[r >> 5], 1u << (r & 31));
    else if (r == -2) atomicOr(&s_bits, GDN_STATUS_POOL_ROW);
  }
  __syncthreads();
  int m = 0, moves = 0;
  auto before = [&](int w) -> unsigned {  // the word's bits of rows before m
    const int k = m - 32 * w;
    return k >= 32 ? ~0u : k <= 0 ? 0u : (1u << k) - 1u;
  };
  if (nwords <= 64) {
    // up to 2 048 rows: every wave forms the whole plan, a word per lane, and the
    // first one writes it: one barrier
    const int w = tid & 63;
    const unsigned live = w < nwords ? map[w] : 0u;
    m = __builtin_amdgcn_readlane(wave_prefix_sum_i(__popc(live)), 63);
    const int both = __popc(live & ~before(w)) | (w < nwords ? __popc(~live & before(w)) << 16 : 0);
    const int inc = wave_prefix_sum_i(both);
    moves = __builtin_amdgcn_readlane(inc, 63) & 0xFFFF;
    if (tid < nwords) {
      movers[w] = (inc - both) & 0xFFFF;
      holes[w] = (inc - both) >> 16;
    }
    __syncthreads();
  } else {
    // a thread owns `per` consecutive words
    const int per = (nwords + kThreads - 1) / kThreads;
    const int w0 = min(tid * per, nwords), w1 = min(w0 + per, nwords);
    int n = 0;
    for (int w = w0; w < w1; ++w) n += __popc(map[w]);
    block_prefix(n, sh);
    m = sh[0];
    int nm = 0, nh = 0;
    for (int w = w0; w < w1; ++w) {
      nm += __popc(map[w] & ~before(w));
      nh += __popc(~map[w] & before(w));
    }
    int pm = block_prefix(nm, sh);
    moves = sh[0];
    int ph = block_prefix(nh, sh);
    for (int w = w0; w < w1; ++w) {
      movers[w] = pm;
      holes[w] = ph;
      pm += __popc(map[w] & ~before(w));
      ph += __popc(~map[w] & before(w));
    }
    __syncthreads();
  }
  // last word whose count of earlier rows is <= k, and the row in it
  auto word_of = [&](const int *pre, int k) {
    int lo = 0, hi = nwords - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= k) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  auto hole_row = [&](int k) {
    const int w = word_of(holes, k);
    return 32 * w + nth_bit(~map[w] & before(w), k - holes[w]);
  };
  auto mover_row = [&](int k) {
    const int w = word_of(movers, k);
    return 32 * w + nth_bit(map[w] & ~before(w), k - movers[w]);
  };
  auto place = [&](int r) {  // where live row r ends up
    if (r < m) return r;
    const int w = r >> 5;
    return hole_row(movers[w] + __popc(map[w] & ~before(w) & ((1u << (r & 31)) - 1u)));
  };

  // renaming, spread over all workgroups
  const int64_t gt = (int64_t)blockIdx.x * kThreads + tid, gn = (int64_t)gridDim.x * kThreads;
  for (int64_t i = gt; i < a.count; i += gn) {
    const int64_t raw = load_index_any(a.dst_rows, a.rows_type, i);
    const int64_t r = raw >= 0 && raw < a.dst_pool ? (int64_t)place((int)raw) : raw;
    if (a.rows_type == GDN_I64) ((int64_t *)a.new_rows)[i] = r;
    else ((int32_t *)a.new_rows)[i] = (int32_t)r;
  }
  if (a.row_map)
    for (int64_t r = gt; r < a.dst_pool; r += gn)
      a.row_map[r] = map[r >> 5] >> (r & 31) & 1 ? place((int)r) : -1;
  if (blockIdx.x == 0 && tid == 0) {
    a.num_live[0] = m;
    if (a.status) a.status[0] = (int32_t)s_bits;
  }

  const auto always = []() { return true; };
  for (unsigned unit = blockIdx.x; unit < u.total; unit += gridDim.x) {
    const int64_t k0 = (int64_t)(unit / u.slices) * u.group, e0 = unit % u.slices * u.slice;
    const int64_t e1 = e0 + u.slice < a.row ? e0 + u.slice : a.row;
    if (k0 >= moves) break;  // units of one group after another: none left
    if (u.group == 1) {
      move_equal<false>(a, __builtin_amdgcn_readfirstlane(mover_row((int)k0)),
                        __builtin_amdgcn_readfirstlane(hole_row((int)k0)), e0, e1, always);
      continue;
    }
    const int cnt = (int)(moves - k0 < u.group ? moves - k0 : u.group);
    __syncthreads();
    if (tid < cnt) {
      s_src[tid] = mover_row((int)k0 + tid);
      s_dst[tid] = hole_row((int)k0 + tid);
    }
    __syncthreads();
    for (int p = 0; p < cnt; ++p) move_equal<false>(a, s_src[p], s_dst[p], e0, e1, always);
  }
}

}  // namespace

static size_t status_map_bytes(const PoolArgs &a) {
  return a.status ? (size_t)((a.dst_pool + 31) / 32) * 4 : 0;
}

template <typename MOVE>
static hipError_t launch_list(const PoolArgs &a, hipStream_t s) {
  const Units u = cut(a, a.count);
  const unsigned grid = unit_grid(a, u) + (a.status ? 1u : 0u);  // one for the status word
  if (grid == 0) return hipSuccess;
  pool_list_kernel<MOVE><<<dim3(grid), dim3(kThreads), status_map_bytes(a), s>>>(a, u);
  return hipGetLastError();
}

template <typename S, typename D>
static hipError_t launch_types(const PoolArgs &a, hipStream_t s) {
  if constexpr (std::is_same<S, D>::value) return launch_list<MoveEqual<false>>(a, s);
  else return launch_list<MoveConvert<S, D>>(a, s);
}

template <typename S>
static hipError_t launch_from(const PoolArgs &a, hipStream_t s) {
  switch (a.dst_dtype) {
    case GDN_F32: return launch_types<S, float>(a, s);
    case GDN_BF16: return launch_types<S, bf16>(a, s);
    case GDN_F16: return launch_types<S, f16>(a, s);
    case GDN_FP8_E4M3: return launch_types<S, fp8e4m3>(a, s);
    default: return launch_types<S, fp8e5m2>(a, s);
  }
}

hipError_t launch_pool_copy(const PoolArgs &a, hipStream_t s) {
  switch (a.src_dtype) {
    case GDN_F32: return launch_from<float>(a, s);
    case GDN_BF16: return launch_from<bf16>(a, s);
    case GDN_F16: return launch_from<f16>(a, s);
    case GDN_FP8_E4M3: return launch_from<fp8e4m3>(a, s);
    default: return launch_from<fp8e5m2>(a, s);
  }
}
hipError_t launch_pool_reset(const PoolArgs &a, hipStream_t s) {
  return launch_list<MoveEqual<true>>(a, s);
}

hipError_t launch_pool_compact(const PoolArgs &a, hipStream_t s) {
  // a mover lies at or behind the new end and its hole before it
  const int64_t entries = a.count < a.dst_pool / 2 ? a.count : a.dst_pool / 2;
  const Units u = cut(a, entries);
  const unsigned want = unit_grid(a, u);
  const int nwords = (int)((a.dst_pool + 31) / 32);
  const int lds = 12 * nwords;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = set_dynamic_lds((const void *)pool_compact_kernel,
                                       12 * (GDN_POOL_MAX_ROWS / 32), done);
  if (e != hipSuccess) return e;
  pool_compact_kernel<<<dim3(want ? want : 1u), dim3(kThreads), lds, s>>>(a, u, nwords);
  return hipGetLastError();
}

}  // namespace gdn
