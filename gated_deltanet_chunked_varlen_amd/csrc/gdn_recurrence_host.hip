// gdn_recurrence_host.hip -- host side of the gated linear recurrence and of
// the state-pool row operators: argument checks, workspace layout, launches.
// Nothing here reads device memory or synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "../../include/gdn_prefill.h"
#include "gdn_internal.h"
#include "gdn_recurrence.h"

using namespace gdn;

uint32_t gdn::rec_wait_limit = 1u << 20;

// Workgroups per channel block for the empty sequences, whose states a pass
// copies: 64 sequences each, at most 64 of them, and no more than the grid
// holds beside the scan's `units` (a grid has fewer than 2^32 threads, and a
// scan's workgroup 512; one fits always: units < 2^22 and ncb <= 2^21).
int32_t gdn::rec_empties(uint32_t units, int32_t ncb, int32_t num_seqs) {
  const int64_t room = ((int64_t)(1 << 23) - 1 - units) / ncb;
  return (int32_t)std::min<int64_t>(std::min<int64_t>(64, room), ((int64_t)num_seqs + 63) / 64);
}

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxUnits = (1 << 22) - 1;  // tiles of 64 tokens x 256 channels
constexpr int64_t kMaxTokens = INT32_MAX - 64;
// sequences: what a kernel's 32-bit loops can step behind without an overflow
constexpr int64_t kMaxSeqs = (int64_t)1 << 30;
constexpr int64_t kMaxDecodeThreads = ((int64_t)1 << 32) - 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool float_type(int d) { return d == GDN_F32 || d == GDN_BF16 || d == GDN_F16; }
bool state_type(int d) { return float_type(d) || d == GDN_FP8_E4M3 || d == GDN_FP8_E5M2; }
bool index_type(int t) { return t == GDN_I32 || t == GDN_I64; }
int64_t size_of(int d) { return d == GDN_F32 ? 4 : d == GDN_BF16 || d == GDN_F16 ? 2 : 1; }

bool aligned(const void *p, int64_t n) { return (uintptr_t)p % (uintptr_t)n == 0; }

enum Mode { kForward = 0, kBackward = 1, kDecode = 2 };

int64_t tiles_of(const gdn_recurrence_params *p, bool backward) {
  const int64_t tile =
      backward ? kRecTile : rec_forward_tile(p->x_dtype, p->g_per_head);
  return std::max<int64_t>(1, (p->total_tokens + tile - 1) / tile);
}

int check_shape(const gdn_recurrence_params *p, int mode) {
  if (!p) return GDN_ERR_NULL;
  if (p->total_tokens < 0 || p->total_tokens > kMaxTokens || p->num_seqs < 0 ||
      p->num_seqs > kMaxSeqs)
    return GDN_ERR_SHAPE;
  if (p->num_heads < 1 || p->head_size < 1) return GDN_ERR_SHAPE;
  const int64_t C = (int64_t)p->num_heads * p->head_size;
  if (C > INT32_MAX / 4) return GDN_ERR_SHAPE;
  if (mode == kDecode) {
    if (p->total_tokens != p->num_seqs || p->cu_seqlens) return GDN_ERR_SHAPE;
    // one thread per four channels of a sequence, in whole workgroups of 256
    if (((C + 3) / 4) * (int64_t)p->num_seqs > kMaxDecodeThreads) return GDN_ERR_SHAPE;
  } else {
    if (!p->cu_seqlens && p->num_seqs != 1) return GDN_ERR_SHAPE;
    const int64_t ncb = (C + kRecChannels - 1) / kRecChannels;
    // one workgroup per unit; a grid holds fewer than 2^32 threads
    if (tiles_of(p, true) * ncb > kMaxUnits) return GDN_ERR_SHAPE;
  }
  if (!float_type(p->x_dtype)) return GDN_ERR_DTYPE;
  if (p->g_dtype != GDN_F32 && p->g_dtype != p->x_dtype) return GDN_ERR_DTYPE;
  if (p->g_per_head != 0 && p->g_per_head != 1) return GDN_ERR_SHAPE;
  if (p->g_per_head && p->head_size != 32 && p->head_size != 64 && p->head_size != 128)
    return GDN_ERR_SHAPE;
  return GDN_OK;
}

struct RecLayout {
  size_t ticket, words, bos, chunk, total;
  bool chain, starts, own_chunk;
};

// The chain's tickets and words (more than one tile), the sequence starts of a
// batch that does not fit a wave's lanes, and the backward pass's states where
// the caller kept none.
RecLayout plan(const gdn_recurrence_params *p, bool backward) {
  RecLayout L{};
  const int64_t C = (int64_t)p->num_heads * p->head_size, tiles = tiles_of(p, backward);
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off = align_up(off + bytes); return o; };
  L.chain = tiles > 1;
  L.starts = p->num_seqs > kDirectSeqs;
  L.own_chunk = backward && !p->chunk_states && tiles > 1;
  if (L.chain) {
    const int64_t ncb = (C + kRecChannels - 1) / kRecChannels;
    L.ticket = take((size_t)ncb * kTicketStep * sizeof(uint32_t));
    L.words = take((size_t)(tiles + groups_of(tiles)) * C * sizeof(unsigned long long));
  }
  if (L.starts) L.bos = take(sizeof(int32_t) * ((size_t)p->num_seqs + 1));
  // rows of 64 tokens, the backward pass's tiles
  if (L.own_chunk) L.chunk = take((size_t)tiles * C * sizeof(float));
  L.total = off;
  return L;
}

// A token or row stride: 0 (contiguous) or at least the length of a row.
bool stride_ok(int64_t s, int64_t row) { return s == 0 || s >= row; }

int validate(const gdn_recurrence_params *p, int mode) {
  int rc = check_shape(p, mode);
  if (rc != GDN_OK) return rc;
  const int64_t T = p->total_tokens, N = p->num_seqs;
  const int64_t C = (int64_t)p->num_heads * p->head_size;
  const int64_t grow = p->g_per_head ? p->num_heads : C;
  const int64_t xs = size_of(p->x_dtype), gs = size_of(p->g_dtype);
  if (T > 0 && (!p->x || !p->g)) return GDN_ERR_NULL;
  if (!stride_ok(p->x_stride, C) || !stride_ok(p->g_stride, grow)) return GDN_ERR_STRIDES;
  if (!aligned(p->x, xs) || !aligned(p->g, gs)) return GDN_ERR_ALIGN;
  if (p->cu_seqlens && !index_type(p->cu_seqlens_type)) return GDN_ERR_DTYPE;
  if (p->initial_state) {
    if (!state_type(p->initial_state_dtype)) return GDN_ERR_DTYPE;
    if (!stride_ok(p->initial_state_stride, C)) return GDN_ERR_STRIDES;
    if (!aligned(p->initial_state, size_of(p->initial_state_dtype))) return GDN_ERR_ALIGN;
  }
  if (p->state_indices) {
    if (mode == kBackward) return GDN_ERR_STATE;
    if (!index_type(p->state_indices_type)) return GDN_ERR_DTYPE;
    if (p->pool_size < 1) return GDN_ERR_STATE;
  }
  if (mode == kBackward) {
    if (T > 0 && (!p->doutput || !p->dx || !p->dg)) return GDN_ERR_NULL;
    if (!stride_ok(p->doutput_stride, C)) return GDN_ERR_STRIDES;
    if (!aligned(p->doutput, xs) || !aligned(p->dx, xs) || !aligned(p->dg, gs) ||
        !aligned(p->dfinal_state, 4) || !aligned(p->dinitial_state, 4))
      return GDN_ERR_ALIGN;
  } else {
    if (T > 0 && !p->output) return GDN_ERR_NULL;
    if (!aligned(p->output, xs)) return GDN_ERR_ALIGN;
    if (p->output_final_state) {
      if (!p->output_state && N > 0) return GDN_ERR_STATE;
      if (!state_type(p->output_state_dtype)) return GDN_ERR_DTYPE;
      if (!stride_ok(p->output_state_stride, C)) return GDN_ERR_STRIDES;
      if (!aligned(p->output_state, size_of(p->output_state_dtype))) return GDN_ERR_ALIGN;
    }
  }
  if (mode == kDecode) {
    if (p->chunk_states) return GDN_ERR_STATE;
    return GDN_OK;
  }
  if (!aligned(p->chunk_states, 4)) return GDN_ERR_ALIGN;
  const size_t need = plan(p, mode == kBackward).total;
  if (p->workspace_bytes < need || (need > 0 && !p->workspace)) return GDN_ERR_WORKSPACE;
  if (need > 0 && !aligned(p->workspace, kAlign)) return GDN_ERR_ALIGN;
  return GDN_OK;
}

void fill(const gdn_recurrence_params *p, int num_cus, RecArgs &a) {
  std::memset(&a, 0, sizeof(a));
  const int64_t C = (int64_t)p->num_heads * p->head_size;
  a.T = p->total_tokens;
  a.N = p->num_seqs;
  a.H = p->num_heads;
  a.D = p->head_size;
  a.C = (int32_t)C;
  a.x_dtype = p->x_dtype;
  a.g_dtype = p->g_dtype;
  a.g_per_head = p->g_per_head;
  a.x = p->x;
  a.g = p->g;
  a.x_stride = p->x_stride ? p->x_stride : C;
  a.g_stride = p->g_stride ? p->g_stride : (p->g_per_head ? p->num_heads : C);
  a.cu = p->cu_seqlens;
  a.cu_type = p->cu_seqlens_type;
  a.init = p->initial_state;
  a.init_dtype = p->initial_state_dtype;
  a.init_stride = p->initial_state_stride ? p->initial_state_stride : C;
  a.sidx = p->state_indices;
  a.sidx_type = p->state_indices_type;
  a.pool_rows = p->pool_size;
  a.status = p->status;
  a.num_cus = num_cus;
  a.wait_limit = rec_wait_limit;
  a.ncb = (int32_t)((C + kRecChannels - 1) / kRecChannels);
}

// Every row of the tensor is whole aligned groups of four elements.
bool rows_vec(const void *p, int64_t stride, int64_t es) {
  return aligned(p, 4 * es) && stride % 4 == 0;
}

int run_scan(const gdn_recurrence_params *p, bool backward, hipStream_t s) {
  int num_cus = 0;
  const int rc = check_device(&num_cus);
  if (rc != GDN_OK) return rc;
  const RecLayout L = plan(p, backward);
  unsigned char *ws = (unsigned char *)p->workspace;
  RecArgs a;
  fill(p, num_cus, a);
  const int64_t C = a.C, xs = size_of(p->x_dtype), gs = size_of(p->g_dtype);
  int32_t *bos = nullptr;
  // a pass's tiles, and its chain where there is more than one
  auto cut = [&](RecArgs &r, bool back) {
    r.ntiles = (int32_t)tiles_of(p, back);
    r.units = (uint32_t)r.ntiles * (uint32_t)r.ncb;
    if (r.ntiles > 1) {
      r.ticket = (uint32_t *)(ws + L.ticket);
      r.words = (unsigned long long *)(ws + L.words);
      r.groups = r.words + (int64_t)r.ntiles * r.C;
    }
  };
  if (L.starts) a.bos = bos = (int32_t *)(ws + L.bos);
  a.chunk = L.own_chunk ? (float *)(ws + L.chunk) : p->chunk_states;
  a.vec = C % 4 == 0 && rows_vec(p->x, a.x_stride, xs) &&
          (p->g_per_head || rows_vec(p->g, a.g_stride, gs));
  hipError_t e = hipSuccess;
  auto prepare = [&](const RecArgs &r) {
    if (e == hipSuccess && (r.ticket || L.starts)) e = launch_rec_prepare(r, bos, s);
  };
  if (!backward || L.own_chunk) {
    RecArgs f = a;
    cut(f, false);
    if (!backward) {
      f.out = p->output;
      f.vec = f.vec && rows_vec(p->output, C, xs);
      if (p->output_final_state) {
        f.fin = p->output_state;
        f.fin_dtype = p->output_state_dtype;
        f.fin_stride = p->output_state_stride ? p->output_state_stride : C;
        // in a pool worked on in place their final states are there already
        const bool same = f.fin == f.init && f.fin_dtype == f.init_dtype &&
                          f.fin_stride == f.init_stride;
        f.empties = f.fin && !same ? rec_empties(f.units, f.ncb, f.N) : 0;
      }
    }
    prepare(f);
    if (e == hipSuccess) e = launch_rec_forward(f, s);
  }
  if (backward) {
    a.dy = p->doutput;
    a.dy_stride = p->doutput_stride ? p->doutput_stride : C;
    a.dfin = p->dfinal_state;
    a.dx = p->dx;
    a.dg = p->dg;
    a.dinit = p->dinitial_state;
    a.vec = a.vec && rows_vec(p->doutput, a.dy_stride, xs) && rows_vec(p->dx, C, xs) &&
            (p->g_per_head || rows_vec(p->dg, C, gs));
    cut(a, true);
    a.empties = a.dinit ? rec_empties(a.units, a.ncb, a.N) : 0;
    prepare(a);
    if (e == hipSuccess) e = launch_rec_backward(a, s);
  }
  return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

// ---------------------------------------------------------------------- pools

bool pool_strides_ok(const int64_t s[4], int64_t rows, const int64_t ext[3]) {
  if (s[0] == 0 && s[1] == 0 && s[2] == 0 && s[3] == 0) return true;
  const int64_t n[4] = {rows, ext[0], ext[1], ext[2]};
  int idx[4] = {0, 1, 2, 3};
  for (int i = 0; i < 4; ++i)
    if (s[i] <= 0 && n[i] > 1) return false;
  std::sort(idx, idx + 4, [&](int x, int y) { return s[x] < s[y]; });
  int64_t reach = 1;  // elements spanned by the dimensions so far
  for (int k = 0; k < 4; ++k) {
    if (n[idx[k]] <= 1) continue;  // never overlaps anything
    if (s[idx[k]] < reach) return false;
    reach = s[idx[k]] * (n[idx[k]] - 1) + reach;
  }
  return true;
}

void pool_strides(const int64_t in[4], const int64_t ext[3], int64_t out[4]) {
  if (in[0] == 0 && in[1] == 0 && in[2] == 0 && in[3] == 0) {
    out[3] = 1;
    out[2] = ext[2];
    out[1] = ext[1] * ext[2];
    out[0] = ext[0] * ext[1] * ext[2];
  } else {
    for (int i = 0; i < 4; ++i) out[i] = in[i];
  }
}

// Bytes from a row's first element to behind its last.
int64_t row_span(const int64_t s[4], const int64_t ext[3], int64_t es) {
  return (1 + (ext[0] - 1) * s[1] + (ext[1] - 1) * s[2] + (ext[2] - 1) * s[3]) * es;
}

bool row_contiguous(const int64_t s[4], const int64_t ext[3]) {
  return (ext[2] == 1 || s[3] == 1) && (ext[1] == 1 || s[2] == ext[2]) &&
         (ext[0] == 1 || s[1] == ext[1] * ext[2]);
}

// One dimension of two views: the distance in bytes from an index of the one to
// the next, and the range of (source index - destination index).
struct Steps {
  int64_t bytes, lo, hi;
};

// Some element of the source view (ss bytes, the first at byte `at`) and some of
// the destination view (ds bytes, the first at byte 0) share a byte.  The
// dimensions go from the longest step to the shortest; as a view's elements do
// not overlap, few differences come into question in each.
bool meet(int64_t at, const Steps *d, int n, int64_t ss, int64_t ds) {
  if (n == 0) return -ss < at && at < ds;
  int64_t below = 0, above = 0;  // what the shorter steps can add
  for (int k = 1; k < n; ++k) {
    below += d[k].lo * d[k].bytes;
    above += d[k].hi * d[k].bytes;
  }
  // -ss < at + i * bytes + (below .. above) < ds
  const int64_t from = std::max(d->lo, (-ss - at - above) / d->bytes - 1);
  const int64_t to = std::min(d->hi, (ds - at - below) / d->bytes + 1);
  for (int64_t i = from; i <= to; ++i)
    if (meet(at + i * d->bytes, d + 1, n - 1, ss, ds)) return true;
  return false;
}

// The two views share no byte: their rows do not meet as whole stretches, or
// where they are interleaved closer than that, their elements do not.  False
// also where the views' steps differ, so that this is not settled.
bool views_apart(int64_t at, const int64_t ss[4], int64_t srows, int64_t se, const int64_t ds[4],
                 int64_t drows, int64_t de, const int64_t ext[3]) {
  Steps d[4];
  int n = 0;
  auto dim = [&](int64_t s, int64_t sn, int64_t t, int64_t tn) {
    s *= se;
    t *= de;
    if (sn > 1 && tn > 1 && s != t) return false;
    if (sn > 1 || tn > 1) d[n++] = {sn > 1 ? s : t, 1 - tn, sn - 1};
    return true;
  };
  if (!dim(ss[0], srows, ds[0], drows)) return false;
  if (!meet(at, d, n, row_span(ss, ext, se), row_span(ds, ext, de))) return true;
  for (int i = 0; i < 3; ++i)
    if (!dim(ss[i + 1], ext[i], ds[i + 1], ext[i])) return false;
  std::sort(d, d + n, [](const Steps &x, const Steps &y) { return x.bytes > y.bytes; });
  return !meet(at, d, n, se, de);
}

struct PoolPlan {
  int64_t src_str[4], dst_str[4];
  bool same, flat;
  int align;
};

enum PoolMode { kCopy = 0, kReset = 1, kCompact = 2 };

// Checks a pool call and settles its strides and access width.
int pool_plan(const gdn_pool_params *p, int mode, PoolPlan &L) {
  if (!p) return GDN_ERR_NULL;
  int64_t row = 1;
  for (int i = 0; i < 3; ++i) {
    if (p->extent[i] < 1 || p->extent[i] > INT32_MAX) return GDN_ERR_SHAPE;
    row *= p->extent[i];
    if (row > (int64_t)1 << 40) return GDN_ERR_SHAPE;
  }
  if (p->dst_pool_rows < 0 || p->dst_pool_rows > GDN_POOL_MAX_ROWS) return GDN_ERR_SHAPE;
  if (p->count < 0 || p->count > INT32_MAX) return GDN_ERR_SHAPE;
  if (!state_type(p->dst_dtype) || !index_type(p->rows_type)) return GDN_ERR_DTYPE;
  if (p->count > 0 && !p->dst_rows) return GDN_ERR_NULL;
  if (p->dst_pool_rows > 0 && !p->dst) return GDN_ERR_NULL;
  const int64_t ds = size_of(p->dst_dtype);
  if (!aligned(p->dst, ds)) return GDN_ERR_ALIGN;
  if (!pool_strides_ok(p->dst_strides, p->dst_pool_rows, p->extent)) return GDN_ERR_STRIDES;
  pool_strides(p->dst_strides, p->extent, L.dst_str);
  L.flat = row_contiguous(L.dst_str, p->extent);
  L.same = false;
  // (a pool of one row is never stepped over, whatever its row stride)
  auto width = [&](const void *base, int64_t rows, const int64_t s[4], int64_t es) {
    const int64_t step = rows > 1 ? s[0] * es : 0;
    int64_t w = 16;
    while (w > 1 && ((uintptr_t)base % w || step % w || (row * es) % w)) w /= 2;
    return (int)w;
  };
  L.align = width(p->dst, p->dst_pool_rows, L.dst_str, ds);
  if (mode != kCopy) {
    for (int i = 0; i < 4; ++i) L.src_str[i] = L.dst_str[i];
    return GDN_OK;
  }
  // every entry is compared with every other one (k7_pool.hip)
  if (p->count > GDN_POOL_MAX_ROWS) return GDN_ERR_SHAPE;
  if (p->src_pool_rows < 0 || p->src_pool_rows > GDN_POOL_MAX_ROWS) return GDN_ERR_SHAPE;
  if (!state_type(p->src_dtype)) return GDN_ERR_DTYPE;
  if (p->count > 0 && !p->src_rows) return GDN_ERR_NULL;
  if (!p->src) return GDN_ERR_NULL;
  const int64_t ss = size_of(p->src_dtype);
  if (!aligned(p->src, ss)) return GDN_ERR_ALIGN;
  if (!pool_strides_ok(p->src_strides, p->src_pool_rows, p->extent)) return GDN_ERR_STRIDES;
  pool_strides(p->src_strides, p->extent, L.src_str);
  L.flat = L.flat && row_contiguous(L.src_str, p->extent);
  L.align = std::min(L.align, width(p->src, p->src_pool_rows, L.src_str, ss));
  // the same view, or no shared elements
  bool strides_equal = p->src_dtype == p->dst_dtype;
  for (int i = 0; i < 4; ++i) strides_equal = strides_equal && L.src_str[i] == L.dst_str[i];
  L.same = p->src == p->dst && strides_equal;
  if (!L.same && p->src_pool_rows > 0 && p->dst_pool_rows > 0) {
    const uintptr_t s0 = (uintptr_t)p->src, d0 = (uintptr_t)p->dst;
    const int64_t sr = row_span(L.src_str, p->extent, ss), dr = row_span(L.dst_str, p->extent, ds);
    const uintptr_t s1 = s0 + (uintptr_t)((p->src_pool_rows - 1) * L.src_str[0] * ss + sr);
    const uintptr_t d1 = d0 + (uintptr_t)((p->dst_pool_rows - 1) * L.dst_str[0] * ds + dr);
    // interleaved views of one buffer (the layers of a [rows, layers, ...] pool)
    if (s0 < d1 && d0 < s1 &&
        !views_apart((int64_t)(s0 - d0), L.src_str, p->src_pool_rows, ss, L.dst_str,
                     p->dst_pool_rows, ds, p->extent))
      return GDN_ERR_STATE;
  }
  return GDN_OK;
}

int pool_args(const gdn_pool_params *p, int mode, PoolArgs &a) {
  PoolPlan L;
  int rc = pool_plan(p, mode, L);
  if (rc != GDN_OK) return rc;
  int num_cus = 0;
  rc = check_device(&num_cus);
  if (rc != GDN_OK) return rc;
  std::memset(&a, 0, sizeof(a));
  a.row = p->extent[0] * p->extent[1] * p->extent[2];
  a.d2 = p->extent[1];
  a.d3 = p->extent[2];
  a.src = mode == kCopy ? p->src : mode == kCompact ? p->dst : nullptr;
  a.src_dtype = mode == kCopy ? p->src_dtype : p->dst_dtype;
  a.src_pool = mode == kCopy ? p->src_pool_rows : p->dst_pool_rows;
  a.dst = p->dst;
  a.dst_dtype = p->dst_dtype;
  a.dst_pool = p->dst_pool_rows;
  for (int i = 0; i < 4; ++i) {
    a.src_str[i] = L.src_str[i];
    a.dst_str[i] = L.dst_str[i];
  }
  a.src_rows = p->src_rows;
  a.dst_rows = p->dst_rows;
  a.rows_type = p->rows_type;
  a.count = p->count;
  a.status = p->status;
  a.same = L.same;
  a.flat = L.flat;
  a.align = L.align;
  a.num_cus = num_cus;
  return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_recurrence_workspace_size(const gdn_recurrence_params *p, int32_t backward) {
  if (check_shape(p, backward ? kBackward : kForward) != GDN_OK) return 0;
  return plan(p, backward != 0).total;
}

int gdn_validate_recurrence_host(const gdn_recurrence_params *p, int32_t mode) {
  if (mode < kForward || mode > kDecode) return GDN_ERR_SHAPE;
  return validate(p, mode);
}

int gdn_recurrence(const gdn_recurrence_params *p, void *stream) {
  const int rc = validate(p, kForward);
  return rc != GDN_OK ? rc : run_scan(p, false, (hipStream_t)stream);
}

int gdn_recurrence_backward(const gdn_recurrence_params *p, void *stream) {
  const int rc = validate(p, kBackward);
  return rc != GDN_OK ? rc : run_scan(p, true, (hipStream_t)stream);
}

int gdn_recurrence_decode(const gdn_recurrence_params *p, void *stream) {
  int rc = validate(p, kDecode);
  if (rc != GDN_OK) return rc;
  int num_cus = 0;
  rc = check_device(&num_cus);
  if (rc != GDN_OK) return rc;
  RecArgs a;
  fill(p, num_cus, a);
  if (a.N == 0 && !a.status) return GDN_OK;
  const int64_t xs = size_of(p->x_dtype), gs = size_of(p->g_dtype);
  a.out = p->output;
  if (p->output_final_state) {
    a.fin = p->output_state;
    a.fin_dtype = p->output_state_dtype;
    a.fin_stride = p->output_state_stride ? p->output_state_stride : a.C;
  }
  a.vec = a.C % 4 == 0 && rows_vec(p->x, a.x_stride, xs) && rows_vec(p->output, a.C, xs) &&
          (p->g_per_head || rows_vec(p->g, a.g_stride, gs));
  return launch_rec_decode(a, (hipStream_t)stream) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int gdn_validate_pool_host(const gdn_pool_params *p, int32_t mode) {
  if (mode < kCopy || mode > kCompact) return GDN_ERR_SHAPE;
  PoolPlan L;
  return pool_plan(p, mode, L);
}

int gdn_pool_copy(const gdn_pool_params *p, void *stream) {
  PoolArgs a;
  const int rc = pool_args(p, kCopy, a);
  if (rc != GDN_OK) return rc;
  return launch_pool_copy(a, (hipStream_t)stream) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int gdn_pool_reset(const gdn_pool_params *p, void *stream) {
  PoolArgs a;
  const int rc = pool_args(p, kReset, a);
  if (rc != GDN_OK) return rc;
  return launch_pool_reset(a, (hipStream_t)stream) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int gdn_pool_compact(const gdn_pool_params *p, void *new_rows, int32_t *num_live,
                     int32_t *row_map, void *stream) {
  PoolArgs a;
  const int rc = pool_args(p, kCompact, a);
  if (rc != GDN_OK) return rc;
  if (!num_live || (p->count > 0 && !new_rows)) return GDN_ERR_NULL;
  const int64_t es = p->rows_type == GDN_I64 ? 8 : 4;
  const uintptr_t n0 = (uintptr_t)new_rows, r0 = (uintptr_t)p->dst_rows;
  const uintptr_t len = (uintptr_t)(p->count * es);
  if (p->count > 0 && n0 < r0 + len && r0 < n0 + len) return GDN_ERR_STATE;
  a.new_rows = new_rows;
  a.num_live = num_live;
  a.row_map = row_map;
  return launch_pool_compact(a, (hipStream_t)stream) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // extern "C"
