// gdn_layers_host.hip -- host side of the short convolution, the selective scan
// and beam search: argument checks, workspace layout, launches.  Nothing here
// reads device memory or synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>
#include <memory>
#include <new>

#include "../../include/gdn_prefill.h"
#include "gdn_layers.h"
#include "gdn_pool_views.h"
#include "gdn_recurrence.h"

using namespace gdn;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxTokens = INT32_MAX - 1024;  // a kernel's 32-bit token numbers
constexpr int64_t kMaxSeqs = (int64_t)1 << 30;
// workgroups of 256 threads in a grid of fewer than 2^32 threads
constexpr int64_t kMaxGrid = (1 << 24) - 1;
constexpr int64_t kUnitBytes = 64 << 10;  // of a row that one workgroup copies

enum Mode { kForward = 0, kBackward = 1, kDecode = 2 };

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool float_type(int d) { return d == GDN_F32 || d == GDN_BF16 || d == GDN_F16; }
bool state_type(int d) { return float_type(d) || d == GDN_FP8_E4M3 || d == GDN_FP8_E5M2; }
bool index_type(int t) { return t == GDN_I32 || t == GDN_I64; }
int64_t size_of(int d) { return d == GDN_F32 ? 4 : d == GDN_BF16 || d == GDN_F16 ? 2 : 1; }
bool aligned(const void *p, int64_t n) { return (uintptr_t)p % (uintptr_t)n == 0; }
bool stride_ok(int64_t s, int64_t row) { return s == 0 || s >= row; }

// Bytes [p, p + rows of `row` elements, `stride` apart) of two tensors meet.
struct Span {
  uintptr_t lo, hi;
  Span(const void *p, int64_t rows, int64_t stride, int64_t row, int64_t es)
      : lo((uintptr_t)p), hi(lo + (p && rows > 0 ? (uintptr_t)(((rows - 1) * stride + row) * es) : 0)) {}
  bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

// What the two sequence operators share of their parameters.
template <typename P> int check_batch(const P *p, int mode, int64_t row) {
  const int64_t N = p->num_seqs;
  if (p->total_tokens < 0 || p->total_tokens > kMaxTokens || N < 0 || N > kMaxSeqs)
    return GDN_ERR_SHAPE;
  if (mode == kDecode ? (p->total_tokens != N || p->cu_seqlens) : (!p->cu_seqlens && N != 1))
    return GDN_ERR_SHAPE;
  if (p->cu_seqlens && !index_type(p->cu_seqlens_type)) return GDN_ERR_DTYPE;
  if (p->initial_state) {
    if (!state_type(p->initial_state_dtype)) return GDN_ERR_DTYPE;
    if (!stride_ok(p->initial_state_stride, row)) return GDN_ERR_STRIDES;
    if (!aligned(p->initial_state, size_of(p->initial_state_dtype))) return GDN_ERR_ALIGN;
  }
  if (p->state_indices) {
    if (mode == kBackward) return GDN_ERR_STATE;
    if (!index_type(p->state_indices_type)) return GDN_ERR_DTYPE;
    if (p->pool_size < 1) return GDN_ERR_STATE;
  }
  if (mode != kBackward && p->output_final_state) {
    if (!p->output_state && N > 0) return GDN_ERR_STATE;
    if (!state_type(p->output_state_dtype)) return GDN_ERR_DTYPE;
    if (!stride_ok(p->output_state_stride, row)) return GDN_ERR_STRIDES;
    if (!aligned(p->output_state, size_of(p->output_state_dtype))) return GDN_ERR_ALIGN;
  }
  return GDN_OK;
}

// `part`: elements of a state's rows of channels.
template <typename P> void fill_batch(const P *p, Batch &b, StateRows &init, StateRows &fin,
                                      int64_t row, int64_t part) {
  auto vec = [&](const StateRows &s) {
    const int64_t es = size_of(s.dtype);
    return aligned(s.p, 16) && s.stride * es % 16 == 0 && part * es % 16 == 0;
  };
  b.T = p->total_tokens;
  b.N = p->num_seqs;
  b.cu = p->cu_seqlens;
  b.cu_type = p->cu_seqlens_type;
  b.sidx = p->state_indices;
  b.sidx_type = p->state_indices_type;
  b.pool_rows = p->pool_size;
  b.status = p->status;
  init.p = const_cast<void *>(p->initial_state);
  init.dtype = p->initial_state_dtype;
  init.stride = p->initial_state_stride ? p->initial_state_stride : row;
  init.vec = vec(init);
  if (p->output_final_state) {
    fin.p = p->output_state;
    fin.dtype = p->output_state_dtype;
    fin.stride = p->output_state_stride ? p->output_state_stride : row;
    fin.vec = vec(fin);
  }
}

// Sequence starts and status of a batch that does not fit a wave's lanes.
hipError_t prepare_batch(Batch &b, int32_t *bos, int num_cus, hipStream_t s) {
  RecArgs r;
  std::memset(&r, 0, sizeof(r));
  r.T = b.T;
  r.N = b.N;
  r.cu = b.cu;
  r.cu_type = b.cu_type;
  r.sidx = b.sidx;
  r.sidx_type = b.sidx_type;
  r.pool_rows = b.pool_rows;
  r.status = b.status;
  r.num_cus = num_cus;
  b.bos = bos;
  return launch_rec_prepare(r, bos, s);
}

struct Taker {
  size_t off = 0;
  size_t operator()(size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes);
    return o;
  }
};

// ---------------------------------------------------------------- convolution

int conv_shape(const gdn_convolution_params *p, int mode) {
  if (!p) return GDN_ERR_NULL;
  if (p->channels < 1 || p->width < 2 || p->width > 4) return GDN_ERR_SHAPE;
  if (!float_type(p->x_dtype)) return GDN_ERR_DTYPE;
  if (p->weight_dtype != GDN_F32 && p->weight_dtype != p->x_dtype) return GDN_ERR_DTYPE;
  if (p->silu != 0 && p->silu != 1) return GDN_ERR_SHAPE;
  const int64_t C = p->channels;
  const int rc = check_batch(p, mode, (p->width - 1) * C);
  if (rc != GDN_OK) return rc;
  if (C > INT32_MAX / 8) return GDN_ERR_SHAPE;
  // a wave per 64 channels of a run of 16 tokens or of a sequence, at the least; in a
  // decode step a workgroup per 256 channels of a sequence
  const int64_t ncb = (C + 63) / 64, T = p->total_tokens, N = p->num_seqs;
  if (mode == kDecode ? (C + 255) / 256 * N > kMaxGrid : ((T + 15) / 16 + N) * ncb > kMaxGrid * 4)
    return GDN_ERR_SHAPE;
  // the sums of dweight and dbias: a workgroup per 32 columns
  if (mode == kBackward && ((p->width + 1) * C + 31) / 32 > kMaxGrid) return GDN_ERR_SHAPE;
  return GDN_OK;
}

struct ConvPlan {
  int vec, run, runs, ncb;
  size_t bos, part, total;
};

// Every row of the tensor is whole aligned groups of 16 bytes.
bool rows16(const void *p, int64_t stride, int64_t es) {
  return aligned(p, 16) && stride * es % 16 == 0;
}

ConvPlan conv_plan(const gdn_convolution_params *p, int mode) {
  ConvPlan L{};
  const int64_t C = p->channels, es = size_of(p->x_dtype), T = p->total_tokens;
  const int64_t V = conv_lane(mode, (int)es);
  // rows of whole 16-byte groups, and a lane's weights too
  L.vec = C * es % 16 == 0 && rows16(p->x, p->x_stride, es) && aligned(p->weight, 16) &&
          aligned(p->bias, 16);
  if (mode == kBackward)
    L.vec = L.vec && rows16(p->doutput, p->doutput_stride, es) && aligned(p->dx, 16);
  else
    L.vec = L.vec && aligned(p->output, 16);
  const int64_t block = 64 * (L.vec ? V : 1);
  L.ncb = (int)((C + block - 1) / block);
  // Long runs read the rows before them less often, short ones fill the GPU: 64
  // tokens from four waves per SIMD (256 CUs) on.
  L.run = 16;
  while (L.run < 64 && (T / (2 * L.run)) * L.ncb >= 4096) L.run *= 2;
  L.runs = (int)((T + L.run - 1) / L.run);
  Taker take;
  if (mode != kDecode && p->num_seqs > kDirectSeqs)
    L.bos = take(sizeof(int32_t) * ((size_t)p->num_seqs + 1));
  if (mode == kBackward) L.part = take(sizeof(float) * (size_t)L.runs * (p->width + 1) * C);
  L.total = take.off;
  return L;
}

// The workspace's size is the larger of both cuts: it does not depend on
// addresses.
size_t conv_bytes(const gdn_convolution_params *p, int mode) {
  gdn_convolution_params q = *p;
  q.x = q.doutput = q.output = q.dx = nullptr;
  q.weight = q.bias = nullptr;
  const size_t vec = conv_plan(&q, mode).total;
  q.x = (const void *)1;
  return std::max(vec, conv_plan(&q, mode).total);
}

int conv_validate(const gdn_convolution_params *p, int mode) {
  const int rc = conv_shape(p, mode);
  if (rc != GDN_OK) return rc;
  const int64_t T = p->total_tokens, C = p->channels;
  const int64_t xs = size_of(p->x_dtype), ws = size_of(p->weight_dtype);
  if (!p->weight || (T > 0 && !p->x)) return GDN_ERR_NULL;
  if (!stride_ok(p->x_stride, C)) return GDN_ERR_STRIDES;
  if (!aligned(p->x, xs) || !aligned(p->weight, ws) || !aligned(p->bias, ws)) return GDN_ERR_ALIGN;
  const Span x(p->x, T, p->x_stride ? p->x_stride : C, C, xs);
  if (mode == kBackward) {
    if (!p->dweight || (T > 0 && (!p->doutput || !p->dx))) return GDN_ERR_NULL;
    if (!stride_ok(p->doutput_stride, C)) return GDN_ERR_STRIDES;
    if (!aligned(p->doutput, xs) || !aligned(p->dx, xs) || !aligned(p->dweight, 4) ||
        !aligned(p->dbias, 4) || !aligned(p->dfinal_state, 4) || !aligned(p->dinitial_state, 4))
      return GDN_ERR_ALIGN;
    const Span dx(p->dx, T, C, C, xs);
    if (dx.meets(x) || dx.meets(Span(p->doutput, T, p->doutput_stride ? p->doutput_stride : C, C, xs)))
      return GDN_ERR_STATE;
  } else {
    if (T > 0 && !p->output) return GDN_ERR_NULL;
    if (!aligned(p->output, xs)) return GDN_ERR_ALIGN;
    // a token's window is read by other workgroups than the token's own; in a decode
    // step a thread reads what it overwrites, if the rows are the same
    const bool same = mode == kDecode && p->output == p->x &&
                      (T <= 1 || p->x_stride == 0 || p->x_stride == C);
    if (!same && Span(p->output, T, C, C, xs).meets(x)) return GDN_ERR_STATE;
  }
  if (mode == kDecode) return GDN_OK;
  const size_t need = conv_bytes(p, mode);
  if (p->workspace_bytes < need || (need > 0 && !p->workspace)) return GDN_ERR_WORKSPACE;
  if (need > 0 && !aligned(p->workspace, kAlign)) return GDN_ERR_ALIGN;
  return GDN_OK;
}

int conv_run(const gdn_convolution_params *p, int mode, hipStream_t s) {
  int num_cus = 0;
  int rc = conv_validate(p, mode);
  if (rc == GDN_OK) rc = check_device(&num_cus);
  if (rc != GDN_OK) return rc;
  const ConvPlan L = conv_plan(p, mode);
  unsigned char *ws = (unsigned char *)p->workspace;
  ConvArgs a;
  std::memset(&a, 0, sizeof(a));
  const int64_t C = p->channels;
  fill_batch(p, a.b, a.init, a.fin, (p->width - 1) * C, C);
  a.C = p->channels;
  a.W = p->width;
  a.x_dtype = p->x_dtype;
  a.w_dtype = p->weight_dtype;
  a.silu = p->silu;
  a.x = p->x;
  a.x_stride = p->x_stride ? p->x_stride : C;
  a.w = p->weight;
  a.bias = p->bias;
  a.out = p->output;
  a.dy = p->doutput;
  a.dy_stride = p->doutput_stride ? p->doutput_stride : C;
  a.dfin = p->dfinal_state;
  a.dx = p->dx;
  a.dw = p->dweight;
  a.db = p->dbias;
  a.dinit = p->dinitial_state;
  a.run = L.run;
  a.runs = L.runs;
  a.ncb = L.ncb;
  a.vec = L.vec;
  a.fvec = C % 4 == 0 && aligned(p->dfinal_state, 16) && aligned(p->dinitial_state, 16);
  if (mode == kBackward) a.part = (float *)(ws + L.part);
  hipError_t e = hipSuccess;
  if (mode == kDecode) {
    if (a.b.N > 0 || a.b.status) e = launch_conv_decode(a, s);
    return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
  if (a.b.N > kDirectSeqs) e = prepare_batch(a.b, (int32_t *)(ws + L.bos), num_cus, s);
  if (e == hipSuccess) e = mode == kBackward ? launch_conv_backward(a, s) : launch_conv_forward(a, s);
  return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

// ----------------------------------------------------------------------- scan

int64_t scan_blocks(const gdn_scan_params *p) {  // of 64 channels
  return (int64_t)p->groups * ((p->channels / p->groups + 63) / 64);
}

// Tokens of a tile.  A pass over tiles forms every state twice; short tiles fill
// the GPU (four waves per SIMD of 256 CUs), long ones leave fewer states in
// memory.  The backward pass keeps a tile's states in LDS, 16 tokens apart, so
// that its tiles have at most 64 tokens of 16 states; the forward pass that
// leaves chunk_states for it uses the same ones.
int64_t scan_tile(const gdn_scan_params *p, bool backward) {
  const int64_t waves = p->total_tokens * scan_blocks(p);
  int64_t most = 256;
  if (backward) most = p->num_states <= 16 ? 64 : p->num_states <= 32 ? 32 : 16;
  // (All are whole runs of the walk, k12_scan_walk.hip, which leaves chunk_states too.)
  int64_t L = 16;
  while (L < most && waves / (2 * L) >= 4096) L *= 2;
  return L;
}

// The forward pass that walks along the tokens, 16 channels a workgroup, and how
// many segments of them: a walk takes 7.4 to 9 us per 256 tokens and 16 states however
// many workgroups there are (up to one per CU; 7.2 with 32 states, 12 with 8), the passes
// over tiles some 35 us and 12 per 256 tokens of 4096 channels.  Both measured, one
// sequence in bf16, walk and tiles (us):
//   16 states  16 384 x 4096: 487, 803    256 x 4096: 14, 43    2816 x 2048: 85, 114
//              1024 x 1024: 35, 51        1024 x 256: 34, 48
//   32 and 64 states  4096 x 4096: 233, 347 and 606, 1069    8 states  4096 x 2048: 100, 88
// The rule counts a walk at its length without segments: how even these are is not
// known here.
int64_t walk_blocks(const gdn_scan_params *p) {
  return (int64_t)p->groups * ((p->channels / p->groups + 15) / 16);
}
// (It takes 8, 16, 32 or 64 states, in aligned fp32 rows, and aligned B and C.)
int scan_walks(const gdn_scan_params *p) {
  const int64_t xs = size_of(p->x_dtype);
  auto states_ok = [&](const void *q, int dtype, int64_t stride) {
    return !q || (dtype == GDN_F32 && aligned(q, 16) && stride % 4 == 0);
  };
  if (p->num_states != scan_states(p->num_states) || !rows16(p->B, p->b_stride, xs) ||
      !rows16(p->C, p->c_stride, xs) || !aligned(p->A, 4) || p->channels > (1 << 23) ||
      !states_ok(p->initial_state, p->initial_state_dtype, p->initial_state_stride) ||
      (p->output_final_state &&
       !states_ok(p->output_state, p->output_state_dtype, p->output_state_stride)))
    return 0;
  const int64_t steps = (p->total_tokens + 255) / 256, n = scan_states(p->num_states);
  // us, times 16 states and 4096 channels
  const int64_t walk = 9 * steps * n * 4096;
  const int64_t tiles = 35 * 16 * 4096 + 12 * steps * n * 64 * scan_blocks(p);
  if (p->total_tokens == 0 || walk > tiles) return 0;
  return (int)std::max<int64_t>(1, std::min<int64_t>(256 / walk_blocks(p),
                                                     std::min<int64_t>(p->num_seqs, steps)));
}

int scan_shape(const gdn_scan_params *p, int mode) {
  if (!p) return GDN_ERR_NULL;
  const int64_t C = p->channels, T = p->total_tokens;
  if (C < 1 || p->num_states < 1 || p->num_states > 64 || p->groups < 1 || C % p->groups != 0)
    return GDN_ERR_SHAPE;
  if (C > (1 << 24)) return GDN_ERR_SHAPE;
  if (!float_type(p->x_dtype)) return GDN_ERR_DTYPE;
  if (p->delta_softplus != 0 && p->delta_softplus != 1) return GDN_ERR_SHAPE;
  const int rc = check_batch(p, mode, C * p->num_states);
  if (rc != GDN_OK) return rc;
  if (mode == kDecode) {
    // a workgroup per 256 lanes of four states (or of a channel) of a sequence
    const int64_t lanes = C * ((p->num_states + 3) / 4);
    return (lanes + 255) / 256 * p->num_seqs > kMaxGrid ? GDN_ERR_SHAPE : GDN_OK;
  }
  if (T > 0 && (walk_blocks(p) + 8) * (16 + 64) > kMaxGrid / 4) return GDN_ERR_SHAPE;
  if (T > 0 && ((T + 15) / 16 + 64) * ((scan_blocks(p) + 3) / 4) > kMaxGrid) return GDN_ERR_SHAPE;
  // the sums of dA, dD and ddelta_bias: a workgroup per 32 columns (of fewer channels
  // where there are tokens)
  if (mode == kBackward && ((p->num_states + 2) * C + 31) / 32 > kMaxGrid) return GDN_ERR_SHAPE;
  const int64_t rows = (int64_t)p->groups * 2 * scan_states(p->num_states);
  if (((T + 255) / 256 * 256) * rows > kMaxGrid * 256) return GDN_ERR_SHAPE;
  return GDN_OK;
}

struct ScanPlan {
  int64_t L, ntiles, Tp;
  size_t bos, bc, a2, chunk, span, flag, start, bct, gchunk, gspan, gflag, psum, pbc, total;
  bool own_chunk;
  int walk;  // segments of the walk, 0: passes over tiles
};

// The workspace is that of the passes over tiles, whichever form the addresses lead
// to: its size does not depend on them.  The walk uses the sequence starts alone.
ScanPlan scan_plan(const gdn_scan_params *p, int mode) {
  ScanPlan S{};
  const bool back = mode == kBackward;
  const int64_t C = p->channels, N = p->num_states, T = p->total_tokens, ns = scan_states(p->num_states);
  S.L = scan_tile(p, back || p->chunk_states);
  S.ntiles = (T + S.L - 1) / S.L;
  S.Tp = S.ntiles * S.L;
  S.own_chunk = S.ntiles > 1 && !p->chunk_states;
  S.walk = back ? 0 : scan_walks(p);
  Taker take;
  if (p->num_seqs > kDirectSeqs) S.bos = take(4 * ((size_t)p->num_seqs + 1));
  S.bc = take(4 * (size_t)T * p->groups * 2 * ns);
  S.a2 = take(4 * (size_t)ns * C);
  const size_t state = 4 * (size_t)S.ntiles * N * C;
  if (S.own_chunk) S.chunk = take(state);
  if (S.ntiles > 1 && (!back || S.own_chunk)) {
    S.span = take(4 * (size_t)S.ntiles * C);
    S.flag = take(4 * (size_t)S.ntiles);
    S.start = take(state);
  }
  if (back) {
    S.bct = take(4 * (size_t)p->groups * 2 * ns * S.Tp);
    if (S.ntiles > 1) {
      S.gchunk = take(state);
      S.gspan = take(4 * (size_t)S.ntiles * C);
      S.gflag = take(4 * (size_t)S.ntiles);
    }
    S.psum = take(4 * (size_t)S.ntiles * (N + 2) * C);
    S.pbc = take(4 * (size_t)scan_blocks(p) * 2 * ns * S.Tp);
  }
  S.total = take.off;
  return S;
}

int scan_validate(const gdn_scan_params *p, int mode) {
  const int rc = scan_shape(p, mode);
  if (rc != GDN_OK) return rc;
  const int64_t T = p->total_tokens, C = p->channels, xs = size_of(p->x_dtype);
  const int64_t bn = (int64_t)p->groups * p->num_states;
  if (!p->A || (T > 0 && (!p->x || !p->delta || !p->B || !p->C))) return GDN_ERR_NULL;
  if (!stride_ok(p->x_stride, C) || !stride_ok(p->delta_stride, C) || !stride_ok(p->z_stride, C) ||
      !stride_ok(p->b_stride, bn) || !stride_ok(p->c_stride, bn))
    return GDN_ERR_STRIDES;
  for (const void *q : {p->x, p->delta, p->z, p->B, p->C})
    if (!aligned(q, xs)) return GDN_ERR_ALIGN;
  for (const void *q : {(const void *)p->A, (const void *)p->D, (const void *)p->delta_bias,
                        (const void *)p->chunk_states})
    if (!aligned(q, 4)) return GDN_ERR_ALIGN;
  auto span = [&](const void *q, int64_t stride, int64_t row) {
    return Span(q, T, stride ? stride : row, row, xs);
  };
  const Span in[6] = {span(p->x, p->x_stride, C), span(p->delta, p->delta_stride, C),
                      span(p->z, p->z_stride, C), span(p->B, p->b_stride, bn),
                      span(p->C, p->c_stride, bn),
                      span(mode == kBackward ? p->doutput : nullptr, p->doutput_stride, C)};
  auto overlaps = [&](const void *q, int64_t row) {
    const Span o = span(q, row, row);
    for (const Span &i : in)
      if (o.meets(i)) return true;
    return false;
  };
  if (mode == kBackward) {
    if (!p->dA || (T > 0 && (!p->doutput || !p->dx || !p->ddelta || !p->dB || !p->dC)))
      return GDN_ERR_NULL;
    if (T > 0 && p->z && !p->dz) return GDN_ERR_NULL;
    if (!stride_ok(p->doutput_stride, C)) return GDN_ERR_STRIDES;
    for (const void *q : {p->doutput, (const void *)p->dx, (const void *)p->ddelta,
                          (const void *)p->dz, (const void *)p->dB, (const void *)p->dC})
      if (!aligned(q, xs)) return GDN_ERR_ALIGN;
    for (const float *q : {(const float *)p->dA, (const float *)p->dD,
                           (const float *)p->ddelta_bias, p->dfinal_state,
                           (const float *)p->dinitial_state})
      if (!aligned(q, 4)) return GDN_ERR_ALIGN;
    if (p->initial_state && p->initial_state_dtype != GDN_F32) return GDN_ERR_DTYPE;
    if (overlaps(p->dx, C) || overlaps(p->ddelta, C) || overlaps(p->dz, C) ||
        overlaps(p->dB, bn) || overlaps(p->dC, bn))
      return GDN_ERR_STATE;
  } else {
    if (T > 0 && !p->output) return GDN_ERR_NULL;
    if (!aligned(p->output, xs)) return GDN_ERR_ALIGN;
    if (overlaps(p->output, C)) return GDN_ERR_STATE;
  }
  if (mode == kDecode) return p->chunk_states ? GDN_ERR_STATE : GDN_OK;
  const size_t need = scan_plan(p, mode).total;
  if (p->workspace_bytes < need || (need > 0 && !p->workspace)) return GDN_ERR_WORKSPACE;
  if (need > 0 && !aligned(p->workspace, kAlign)) return GDN_ERR_ALIGN;
  return GDN_OK;
}

int scan_run(const gdn_scan_params *p, int mode, hipStream_t s) {
  int num_cus = 0;
  int rc = scan_validate(p, mode);
  if (rc == GDN_OK) rc = check_device(&num_cus);
  if (rc != GDN_OK) return rc;
  unsigned char *ws = (unsigned char *)p->workspace;
  ScanArgs a;
  std::memset(&a, 0, sizeof(a));
  const int64_t C = p->channels, bn = (int64_t)p->groups * p->num_states;
  fill_batch(p, a.b, a.init, a.fin, C * p->num_states, C * p->num_states);
  a.C = p->channels;
  a.N = p->num_states;
  a.G = p->groups;
  a.P = p->channels / p->groups;
  a.ncb = (int32_t)scan_blocks(p);
  a.x_dtype = p->x_dtype;
  a.softplus = p->delta_softplus;
  a.x = p->x;
  a.delta = p->delta;
  a.z = p->z;
  a.x_stride = p->x_stride ? p->x_stride : C;
  a.delta_stride = p->delta_stride ? p->delta_stride : C;
  a.z_stride = p->z_stride ? p->z_stride : C;
  a.B = p->B;
  a.C_ = p->C;
  a.b_stride = p->b_stride ? p->b_stride : bn;
  a.c_stride = p->c_stride ? p->c_stride : bn;
  a.A = p->A;
  a.D = p->D;
  a.dbias = p->delta_bias;
  a.out = p->output;
  a.num_cus = num_cus;
  hipError_t e = hipSuccess;
  auto result = [&]() { return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; };
  if (mode == kDecode) {
    const int64_t es = size_of(p->x_dtype);
    a.vec = p->num_states % 4 == 0 && aligned(p->A, 16) && aligned(p->B, 4 * es) &&
            aligned(p->C, 4 * es) && a.b_stride % 4 == 0 && a.c_stride % 4 == 0;
    if (a.b.N > 0 || a.b.status) e = launch_scan_decode(a, s);
    return result();
  }
  const ScanPlan S = scan_plan(p, mode);
  const bool back = mode == kBackward;
  a.L = (int32_t)S.L;
  a.ntiles = (int32_t)S.ntiles;
  a.Tp = S.Tp;
  a.bc = (float *)(ws + S.bc);
  a.a2 = (float *)(ws + S.a2);
  a.chunk = S.own_chunk ? (float *)(ws + S.chunk) : p->chunk_states;
  a.span = (float *)(ws + S.span);
  a.flag = (int32_t *)(ws + S.flag);
  a.start = (float *)(ws + S.start);
  // in a pool worked on in place an empty sequence's final state is there already
  const bool same = a.fin.p == a.init.p && a.fin.dtype == a.init.dtype && a.fin.stride == a.init.stride;
  const bool copies = back ? p->dinitial_state != nullptr : a.fin.p && !same;
  a.empties = copies ? (int32_t)std::min<int64_t>(64, a.b.N) : 0;
  if (a.b.N > kDirectSeqs) e = prepare_batch(a.b, (int32_t *)(ws + S.bos), num_cus, s);
  if (back) {
    a.dy = p->doutput;
    a.dy_stride = p->doutput_stride ? p->doutput_stride : C;
    a.dfin = p->dfinal_state;
    a.dx = p->dx;
    a.ddelta = p->ddelta;
    a.dz = p->dz;
    a.dB = p->dB;
    a.dC = p->dC;
    a.dA = p->dA;
    a.dD = p->dD;
    a.ddbias = p->ddelta_bias;
    a.dinit = p->dinitial_state;
    a.bct = (float *)(ws + S.bct);
    a.gchunk = (float *)(ws + S.gchunk);
    a.gspan = (float *)(ws + S.gspan);
    a.gflag = (int32_t *)(ws + S.gflag);
    a.psum = (float *)(ws + S.psum);
    a.pbc = (float *)(ws + S.pbc);
  }
  if (S.walk) {
    a.chunk = p->chunk_states;  // no states before tiles that nobody asked for
    a.ncb = (int32_t)walk_blocks(p);
    a.nseg = S.walk;
    if (e == hipSuccess) e = launch_scan_walk(a, s);
    return result();
  }
  if (e == hipSuccess) e = launch_scan_prepare(a, s);
  if (e == hipSuccess && a.ntiles > 1 && (!back || S.own_chunk)) e = launch_scan_states(a, s);
  if (e == hipSuccess) e = back ? launch_scan_backward(a, s) : launch_scan_forward(a, s);
  return result();
}

// ----------------------------------------------------------------------- beam

struct BeamPlan {
  int32_t parts, part_len;
  size_t best, where, stat, total;
};

// Parts of a row that a workgroup holds: 8192 logits, or 2048 where that leaves
// fewer than two workgroups per CU.
BeamPlan beam_plan(const gdn_beam_params *p) {
  BeamPlan L{};
  const int64_t rows = (int64_t)p->num_groups * p->num_beams;
  L.part_len = 32 * 256;
  if (rows * ((p->vocab + L.part_len - 1) / L.part_len) < 512) L.part_len = 8 * 256;
  L.parts = (int32_t)((p->vocab + L.part_len - 1) / L.part_len);
  const size_t n = (size_t)rows * L.parts;
  Taker take;
  L.best = take(4 * n * p->num_candidates);
  L.where = take(4 * n * p->num_candidates);
  L.stat = take(8 * n);
  L.total = take.off;
  return L;
}

int beam_shape(const gdn_beam_params *p) {
  if (!p) return GDN_ERR_NULL;
  if (p->num_groups < 0 || p->num_beams < 1 || p->num_beams > GDN_BEAM_MAX || p->vocab < 1 ||
      p->vocab > (1 << 28) || p->num_candidates < 1 || p->num_candidates > GDN_BEAM_MAX ||
      (int64_t)p->num_beams * p->vocab < p->num_candidates)
    return GDN_ERR_SHAPE;
  if ((int64_t)p->num_groups * p->num_beams * ((p->vocab + 2047) / 2048) > kMaxGrid)
    return GDN_ERR_SHAPE;
  if (!float_type(p->logits_dtype)) return GDN_ERR_DTYPE;
  return GDN_OK;
}

int beam_validate(const gdn_beam_params *p) {
  const int rc = beam_shape(p);
  if (rc != GDN_OK) return rc;
  if (!stride_ok(p->logits_stride, p->vocab)) return GDN_ERR_STRIDES;
  if (p->num_groups > 0 &&
      (!p->logits || !p->scores || !p->out_scores || !p->out_parents || !p->out_tokens))
    return GDN_ERR_NULL;
  if (!aligned(p->logits, size_of(p->logits_dtype)) || !aligned(p->scores, 4) ||
      !aligned(p->out_scores, 4) || !aligned(p->out_parents, 4) || !aligned(p->out_tokens, 4))
    return GDN_ERR_ALIGN;
  const size_t need = beam_plan(p).total;
  if (p->workspace_bytes < need || (need > 0 && !p->workspace)) return GDN_ERR_WORKSPACE;
  if (need > 0 && !aligned(p->workspace, kAlign)) return GDN_ERR_ALIGN;
  return GDN_OK;
}

int reorder_pool(const gdn_reorder_params *p, const gdn_reorder_pool &q, ReorderArgs::Pool &o) {
  int64_t row = 1;
  for (int i = 0; i < 3; ++i) {
    if (q.extent[i] < 1 || q.extent[i] > INT32_MAX) return GDN_ERR_SHAPE;
    row *= q.extent[i];
    if (row > (int64_t)1 << 40) return GDN_ERR_SHAPE;
  }
  if (!state_type(q.dtype)) return GDN_ERR_DTYPE;
  if (!q.pool) return GDN_ERR_NULL;
  const int64_t es = size_of(q.dtype);
  if (!aligned(q.pool, es)) return GDN_ERR_ALIGN;
  int64_t s[4];
  if (!pool_strides_ok(q.strides, p->pool_rows, q.extent)) return GDN_ERR_STRIDES;
  pool_strides(q.strides, q.extent, s);
  o.p = (char *)q.pool;
  for (int i = 0; i < 4; ++i) o.str[i] = s[i] * es;
  o.d2 = q.extent[1];
  o.d3 = q.extent[2];
  o.row = row;
  o.es = (int32_t)es;
  o.flat = row_contiguous(s, q.extent);
  const int64_t step = p->pool_rows > 1 ? o.str[0] : 0;
  o.align = 16;
  while (o.align > 1 && ((uintptr_t)q.pool % o.align || step % o.align || (row * es) % o.align))
    o.align /= 2;
  int64_t unit = std::min<int64_t>(kUnitBytes / es, row);
  const int64_t beams = std::max<int64_t>(1, (int64_t)p->num_groups * p->num_beams);
  while ((row + unit - 1) / unit * beams >= kMaxGrid) unit *= 2;  // (and one for the status)
  if (unit > (1 << 30)) return GDN_ERR_SHAPE;
  o.unit = (int32_t)unit;
  o.units = (int32_t)((row + unit - 1) / unit);
  return GDN_OK;
}

// The bytes that a pool lies in, and those of one row.
struct PoolSpan {
  const gdn_reorder_pool *q;
  uintptr_t lo, hi;
  int64_t step, row;  // from row to row
  PoolSpan() = default;
  PoolSpan(const gdn_reorder_pool &pool, int64_t rows) : q(&pool), lo((uintptr_t)pool.pool) {
    int64_t s[4];
    pool_strides(pool.strides, pool.extent, s);
    const int64_t es = size_of(pool.dtype);
    step = s[0] * es;
    row = row_span(s, pool.extent, es);
    hi = lo + (uintptr_t)((rows - 1) * step + row);
  }
  bool apart(const PoolSpan &o, int64_t rows) const {
    if (lo >= o.hi || o.lo >= hi) return true;
    int64_t s[4], t[4];
    pool_strides(q->strides, q->extent, s);
    pool_strides(o.q->strides, o.q->extent, t);
    return views_apart((int64_t)(lo - o.lo), s, rows, size_of(q->dtype), q->extent, t, rows,
                       size_of(o.q->dtype), o.q->extent);
  }
};

// The pools of a call share no bytes.  Where neighbours in memory overlap as
// stretches, they are mostly interleaved row by row (the layers of one buffer):
// then their rows are apart in one period of rows, sorted by their place in it.
// What that does not settle is compared pair by pair.
bool pools_apart(const gdn_reorder_params *p) {
  const int32_t n = p->num_pools;
  const int64_t rows = p->pool_rows;
  if (n < 2 || rows < 1) return true;
  const std::unique_ptr<PoolSpan[]> v(new (std::nothrow) PoolSpan[(size_t)n]);
  auto each_pair = [&](int32_t from, int32_t to) {
    for (int32_t i = from; i < to; ++i)
      for (int32_t j = i + 1; j < to; ++j) {
        const bool ok = v ? v[i].apart(v[j], rows)
                          : PoolSpan(p->pools[i], rows).apart(PoolSpan(p->pools[j], rows), rows);
        if (!ok) return false;
      }
    return true;
  };
  if (!v) return each_pair(0, n);
  for (int32_t i = 0; i < n; ++i) v[i] = PoolSpan(p->pools[i], rows);
  std::sort(&v[0], &v[0] + n, [](const PoolSpan &a, const PoolSpan &b) { return a.lo < b.lo; });
  for (int32_t from = 0, to; from < n; from = to) {
    uintptr_t end = v[from].hi;
    for (to = from + 1; to < n && v[to].lo < end; ++to) end = std::max(end, v[to].hi);
    if (to == from + 1) continue;
    const uintptr_t base = v[from].lo, step = (uintptr_t)v[from].step;
    bool one_step = rows > 1;
    for (int32_t i = from; i < to; ++i)
      one_step = one_step && (uintptr_t)v[i].step == step && (uintptr_t)v[i].row <= step;
    if (one_step) {
      auto place = [&](const PoolSpan &s) { return (s.lo - base) % step; };
      std::sort(&v[0] + from, &v[0] + to,
                [&](const PoolSpan &a, const PoolSpan &b) { return place(a) < place(b); });
      for (int32_t i = from; i < to && one_step; ++i) {
        const uintptr_t next = i + 1 < to ? place(v[i + 1]) : step + place(v[from]);
        one_step = place(v[i]) + (uintptr_t)v[i].row <= next;
      }
      if (one_step) continue;
    }
    if (!each_pair(from, to)) return false;
  }
  return true;
}

int reorder_validate(const gdn_reorder_params *p) {
  if (!p) return GDN_ERR_NULL;
  if (p->num_groups < 0 || p->num_beams < 1 || p->num_beams > GDN_BEAM_MAX || p->num_pools < 1 ||
      p->pool_rows < 0 || p->pool_rows > GDN_POOL_MAX_ROWS)
    return GDN_ERR_SHAPE;
  const int64_t n = (int64_t)p->num_groups * p->num_beams;
  if (n > GDN_POOL_MAX_ROWS) return GDN_ERR_SHAPE;
  if (!index_type(p->index_type)) return GDN_ERR_DTYPE;
  if (!p->pools || (n > 0 && (!p->state_indices || !p->parents || !p->new_indices)))
    return GDN_ERR_NULL;
  const int64_t es = p->index_type == GDN_I64 ? 8 : 4;
  const Span out(p->new_indices, 1, 0, n, es);
  if (out.meets(Span(p->state_indices, 1, 0, n, es)) || out.meets(Span(p->parents, 1, 0, n, es)))
    return GDN_ERR_STATE;
  if (n > 0 && p->pool_rows < 1) return GDN_ERR_STATE;
  for (int32_t i = 0; i < p->num_pools; ++i) {
    ReorderArgs::Pool one;
    const int rc = reorder_pool(p, p->pools[i], one);
    if (rc != GDN_OK) return rc;
  }
  return pools_apart(p) ? GDN_OK : GDN_ERR_STATE;
}

}  // namespace

extern "C" {

size_t gdn_convolution_workspace_size(const gdn_convolution_params *p, int32_t backward) {
  const int mode = backward ? kBackward : kForward;
  return conv_shape(p, mode) == GDN_OK ? conv_bytes(p, mode) : 0;
}
int gdn_validate_convolution_host(const gdn_convolution_params *p, int32_t mode) {
  return mode < kForward || mode > kDecode ? GDN_ERR_SHAPE : conv_validate(p, mode);
}
int gdn_convolution(const gdn_convolution_params *p, void *stream) {
  return conv_run(p, kForward, (hipStream_t)stream);
}
int gdn_convolution_backward(const gdn_convolution_params *p, void *stream) {
  return conv_run(p, kBackward, (hipStream_t)stream);
}
int gdn_convolution_decode(const gdn_convolution_params *p, void *stream) {
  return conv_run(p, kDecode, (hipStream_t)stream);
}

int64_t gdn_scan_chunk(const gdn_scan_params *p) {
  return scan_shape(p, kBackward) == GDN_OK ? scan_tile(p, true) : 0;
}
size_t gdn_scan_workspace_size(const gdn_scan_params *p, int32_t backward) {
  const int mode = backward ? kBackward : kForward;
  return scan_shape(p, mode) == GDN_OK ? scan_plan(p, mode).total : 0;
}
int gdn_validate_scan_host(const gdn_scan_params *p, int32_t mode) {
  return mode < kForward || mode > kDecode ? GDN_ERR_SHAPE : scan_validate(p, mode);
}
int gdn_scan(const gdn_scan_params *p, void *stream) {
  return scan_run(p, kForward, (hipStream_t)stream);
}
int gdn_scan_backward(const gdn_scan_params *p, void *stream) {
  return scan_run(p, kBackward, (hipStream_t)stream);
}
int gdn_scan_decode(const gdn_scan_params *p, void *stream) {
  return scan_run(p, kDecode, (hipStream_t)stream);
}

size_t gdn_beam_workspace_size(const gdn_beam_params *p) {
  return beam_shape(p) == GDN_OK ? beam_plan(p).total : 0;
}
int gdn_validate_beam_host(const gdn_beam_params *p) { return beam_validate(p); }
int gdn_beam_select(const gdn_beam_params *p, void *stream) {
  int rc = beam_validate(p);
  if (rc == GDN_OK) rc = check_device();
  if (rc != GDN_OK || p->num_groups == 0) return rc;
  const BeamPlan L = beam_plan(p);
  unsigned char *ws = (unsigned char *)p->workspace;
  BeamArgs a;
  std::memset(&a, 0, sizeof(a));
  a.B = p->num_groups;
  a.K = p->num_beams;
  a.V = p->vocab;
  a.M = p->num_candidates;
  a.dtype = p->logits_dtype;
  a.logits = p->logits;
  a.stride = p->logits_stride ? p->logits_stride : p->vocab;
  a.scores = p->scores;
  a.out_scores = p->out_scores;
  a.parents = p->out_parents;
  a.tokens = p->out_tokens;
  a.parts = L.parts;
  a.part_len = L.part_len;
  a.best = (float *)(ws + L.best);
  a.where = (int32_t *)(ws + L.where);
  a.stat = (float *)(ws + L.stat);
  const int64_t es = size_of(p->logits_dtype);
  a.vec = rows16(p->logits, a.stride, es) && (int64_t)p->vocab * es % 16 == 0;
  return launch_beam_select(a, (hipStream_t)stream) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int gdn_validate_reorder_host(const gdn_reorder_params *p) { return reorder_validate(p); }
int gdn_pool_reorder(const gdn_reorder_params *p, void *stream) {
  int rc = reorder_validate(p);
  if (rc == GDN_OK) rc = check_device();
  if (rc != GDN_OK) return rc;
  for (int32_t at = 0; at < p->num_pools; at += kReorderPools) {
    ReorderArgs a;
    std::memset(&a, 0, sizeof(a));
    a.B = p->num_groups;
    a.K = p->num_beams;
    a.rows = (int32_t)p->pool_rows;
    a.pools = std::min(kReorderPools, p->num_pools - at);
    a.idx = p->state_indices;
    a.parents = p->parents;
    a.new_idx = at == 0 ? p->new_indices : nullptr;
    a.type = p->index_type;
    a.status = at == 0 ? p->status : nullptr;
    for (int i = 0; i < a.pools; ++i) reorder_pool(p, p->pools[at + i], a.pool[i]);
    if (launch_pool_reorder(a, (hipStream_t)stream) != hipSuccess) return GDN_ERR_LAUNCH;
  }
  return GDN_OK;
}

}  // extern "C"
