/*
 * gdn_prefill.h -- C ABI of libgdn_prefill: the varlen chunked Gated Delta
 * Rule prefill scan on AMD MI355X (gfx950).
 *
 * What is computed (gitcode "FlashInfer GDN Prefill 完全指南", sections
 * "GDN prefill" and "API 全参数解析"; weigao.cc "GDN 与 Chunked Prefill",
 * sections "GDN 是什么" and "块内 state 和块间 final state"): for every
 * sequence i of a packed varlen batch and every sab head h,
 *
 *     S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T
 *     o_t = scale * S_t^T q_t
 *
 * with S a head_size x head_size fp32 state (keys x values) that starts from
 * the given initial state (or zero), is processed in 64-token chunks, and
 * whose final value is optionally written out.  g is alpha itself (the forget
 * gate, default all ones), beta the update gate (default all ones), scale
 * defaults to 1/sqrt(head_size).
 *
 * Conventions shared by every entry point:
 *  - Device pointers unless a comment says "host".  The caller owns every
 *    buffer; the library never allocates, frees or synchronises.  All work is
 *    enqueued on `stream` (a hipStream_t; NULL = the default stream) and the
 *    call returns without waiting.  No device-to-host copy happens in a call.
 *  - Return value: 0 on success, a negative GDN_ERR_* code when a host-side
 *    check fails (then nothing is launched).  gdn_status_string() names codes.
 *  - Data that only the device can check (cu_seqlens contents, state_indices
 *    values, checkpoint_cu_starts contents) never causes an out-of-bounds
 *    access; violations set GDN_STATUS_* bits in the optional device word
 *    `status`, which every call overwrites (it needs no clearing).
 */
#ifndef GDN_PREFILL_H
#define GDN_PREFILL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 2
#define GDN_CHUNK 64 /* kernel chunk length in tokens */

/* Element types.  The two 8-bit float types (OCP FP8 E4M3, max 448, and
 * E5M2, max 57344) are for states only -- initial, final and checkpoint
 * states (gitcode, section "chunk_gated_delta_rule API 全参数解析" lists them
 * for initial_state, section "中间状态检查点" for state_checkpoints).  The
 * pages give no scaling rule for them, so a state is stored by rounding each
 * fp32 element to nearest (ties to even) with saturation at the largest
 * finite value, and read by exact widening. */
typedef enum {
  GDN_F32 = 0, GDN_BF16 = 1, GDN_F16 = 2, GDN_FP8_E4M3 = 3, GDN_FP8_E5M2 = 4
} gdn_dtype;
typedef enum { GDN_I32 = 0, GDN_I64 = 1 } gdn_itype;

/* Host-side error codes (return values). */
#define GDN_OK 0
#define GDN_ERR_NULL -1          /* a required pointer is NULL */
#define GDN_ERR_SHAPE -2         /* token/sequence/head counts or head size */
#define GDN_ERR_HEAD_RATIO -3    /* illegal q/k/v head sharing */
#define GDN_ERR_DTYPE -4         /* unsupported dtype or index type */
#define GDN_ERR_CHECKPOINT -5    /* checkpoint arguments inconsistent */
#define GDN_ERR_STATE -6         /* state / pool arguments inconsistent */
#define GDN_ERR_MAX_SEQLEN -7    /* max_seqlen outside [ceil(T/N), T] */
#define GDN_ERR_WORKSPACE -8     /* workspace missing or too small */
#define GDN_ERR_STRIDES -9       /* state strides not positive/non-overlapping */
#define GDN_ERR_DEVICE -10       /* current device is not gfx950 */
#define GDN_ERR_LAUNCH -11       /* a kernel launch failed */
#define GDN_ERR_ALIGN -12        /* q, k, v or output not 16-byte aligned, or the
                                    workspace not 256-byte aligned (the kernels
                                    move them in 16-byte vector accesses) */
#define GDN_ERR_CP -14          /* use_cp outside {0, 1, 2}, cp_chunk_len not a
                                    non-negative multiple of 64, or GDN_CP_ON
                                    for a call outside the CP domain */
#define GDN_ERR_SCRATCH -13      /* gdn_prefill_noalloc(): the call needs more
                                    workspace than GDN_NOALLOC_SCRATCH_BYTES, or
                                    the static scratch's address is unavailable */

/* Size of the static device scratch that gdn_prefill_noalloc() uses in place
 * of a workspace (one copy per GPU, held until the process ends). */
#define GDN_NOALLOC_SCRATCH_BYTES (128u << 20)

/* Device status bits (written to *status by every call). */
#define GDN_STATUS_CU_SEQLENS 1u        /* cu_seqlens not non-decreasing within [0, T] */
#define GDN_STATUS_CHECKPOINT_STARTS 2u /* checkpoint_cu_starts != prefix sum of floor(len/n) */
#define GDN_STATUS_STATE_INDEX 4u       /* a state index outside [0, pool_size) */
#define GDN_STATUS_CHUNK_CAPACITY 8u    /* more chunks than the sync-free bound (never expected) */
#define GDN_STATUS_POOL_ROW 16u         /* a pool row index outside its pool (-1 is padding, not an error) */
#define GDN_STATUS_POOL_DUPLICATE 32u   /* a destination row named twice (the last entry wins) */
#define GDN_STATUS_POOL_OVERLAP 64u     /* a source row that another entry overwrites (the entry that reads it is skipped) */

/*
 * Parameters of one prefill call (gitcode, section "API 全参数解析"; the
 * fields keep that section's parameter names).
 *
 * Shapes, all row-major and contiguous unless strides are given:
 *   q [T, num_q_heads, D], k [T, num_k_heads, D], v [T, num_v_heads, D],
 *   qkv_dtype F32, BF16 or F16 (gitcode, section "覆盖的公共输入域", names
 *   FP16 and BF16 inputs).  Intermediates are kept in the input type for BF16
 *   and F16 and in fp32 for F32; accumulation is always fp32.
 *   H = num_sab_heads = max(num_q_heads, num_v_heads); legal head sharing:
 *   (hq == hk and hv % hq == 0) or (hk == hv and hq % hk == 0); sab head h
 *   reads q head h / (H / hq), k head h / (H / hk), v head h / (H / hv).
 *   g, beta [T, H] fp32, or NULL for all ones.  g is alpha in (0, 1].
 *   output [T, H, D] in qkv_dtype; rows outside every sequence are untouched.
 *   States are [rows, H, D(v), D(k)]: element [n][h][v][k] is S[k][v]; the
 *   four element strides are given (all zero = contiguous).  initial_state
 *   may be NULL (zero).  state dtypes: F32, BF16, F16, FP8_E4M3 or FP8_E5M2.
 *   state_indices [N] (or NULL): sequence i reads initial_state[idx[i]] and,
 *   if output_final_state, writes output_state[idx[i]]; indices must be
 *   unique (caller precondition, gitcode section "状态池"); output_state may
 *   be the same memory as initial_state (in-place pool); pool_size bounds the
 *   indices and is the row count of both pools.  Without state_indices,
 *   initial_state and output_state have N rows.
 *   checkpoint_every_n_tokens: 0 = off, else a positive multiple of 64;
 *   state_checkpoints [checkpoint_rows, H, D, D] (contiguous; rows outside
 *   [0, checkpoint_rows) are never written) and checkpoint_cu_starts
 *   [N+1] are then both required; checkpoint j (1-based) of sequence i is the
 *   state after j*n of its tokens, at row checkpoint_cu_starts[i] + j - 1.
 *   max_seqlen: 0 = unknown; otherwise must satisfy ceil(T/N) <= max_seqlen
 *   <= T (gitcode section "约束与注意点").
 *   Alignment: q, k, v and output start on 16-byte boundaries and the
 *   workspace on a 256-byte boundary (GDN_ERR_ALIGN otherwise; torch
 *   allocations satisfy both).
 */
typedef struct gdn_prefill_params {
  int64_t total_tokens;   /* T >= 0 */
  int32_t num_seqs;       /* N >= 0; with cu_seqlens NULL, N must be 1 */
  int32_t num_q_heads, num_k_heads, num_v_heads;
  int32_t head_size;      /* D in {32, 64, 128} */
  int32_t qkv_dtype;      /* gdn_dtype */
  const void *q, *k, *v;
  const float *g, *beta;
  int32_t has_scale;
  float scale;
  const void *cu_seqlens; /* [N+1], NULL = one sequence [0, T] */
  int32_t cu_seqlens_type; /* gdn_itype */
  int32_t use_qk_l2norm_in_kernel; /* x / sqrt(sum x^2 + 1e-6), fp32 sums */
  void *output;
  const void *initial_state;
  int32_t initial_state_dtype;
  int64_t initial_state_strides[4];
  int32_t output_final_state;
  void *output_state;
  int32_t output_state_dtype;
  int64_t output_state_strides[4];
  const void *state_indices;
  int32_t state_indices_type;
  int64_t pool_size;
  int32_t checkpoint_every_n_tokens;
  void *state_checkpoints;
  int32_t checkpoint_dtype;
  int64_t checkpoint_rows;
  const void *checkpoint_cu_starts;
  int32_t checkpoint_cu_starts_type;
  int64_t max_seqlen;
  void *workspace;
  size_t workspace_bytes;
  int32_t *status;        /* optional device word */
  /* Context parallelism within the GPU (gitcode, sections "API 全参数解析"
   * (use_cp, _cp_chunk_len, max_seqlen) and "Cake GDN CP 后端" ("四阶段执行
   * 流程"): each sequence is cut into segments of cp_chunk_len tokens, each
   * segment's state transition is formed in parallel, the segment start
   * states are fixed up serially, then every segment runs the ordinary pass
   * from its start state.  use_cp: GDN_CP_AUTO (0) takes it when the call has
   * too few (sequence, head) pairs to fill the GPU and long sequences;
   * GDN_CP_ON (1) requires it and fails closed (GDN_ERR_CP) outside its
   * domain (bf16 / fp16 inputs, head size 128, at most 63 sequences);
   * GDN_CP_OFF (2) never takes it.  cp_chunk_len: 0 = chosen from the shape
   * and max_seqlen (or total_tokens), else a positive multiple of 64 (for
   * tests and tuning).  The results are those of the non-CP pass up to
   * floating-point rounding. */
  int32_t use_cp;
  int64_t cp_chunk_len;
} gdn_prefill_params;

#define GDN_CP_AUTO 0
#define GDN_CP_ON 1
#define GDN_CP_OFF 2

/* ABI version (GDN_ABI_VERSION). */
int gdn_abi_version(void);

/* Static text for an error code (negative) or a status bit (positive). */
const char *gdn_status_string(int code);

/* Upper bound on the number of 64-token chunks of any batch with T tokens
 * and N sequences, needing no look at cu_seqlens:
 * floor((T + 63 * min(N, T)) / 64).  Host only. */
int64_t gdn_max_chunks(int64_t total_tokens, int32_t num_seqs);

/* Bytes of device workspace gdn_prefill() needs for these parameters (only
 * the shape fields are read: token, sequence and head counts, head size,
 * qkv dtype).  The pages' call allocates its scratch internally (gitcode,
 * section "内部机制：plan 缓存、地址重绑定与 CUDA Graph": a cached plan
 * holds the scratch of a shape); here the caller owns it, sized by this
 * function, so a call never allocates.  Host only; 0 for an invalid shape. */
size_t gdn_prefill_workspace_size(const gdn_prefill_params *p);

/* Every host-side check of gdn_prefill() except the device check, without
 * touching the GPU: the argument rules of gitcode, sections "API 全参数解析"
 * (shapes, dtypes, head sharing, defaults), "状态池" (state_indices needs
 * output_state and pool_size), "中间状态检查点" (n a multiple of 64, the two
 * checkpoint buffers given together) and "约束与注意点" (max_seqlen within
 * [ceil(T/N), T]), plus the workspace size and alignment.  Reads only the
 * parameter block, never device memory.  Returns GDN_OK or the GDN_ERR_*
 * code of the first failed check. */
int gdn_validate_host(const gdn_prefill_params *p);

/* The whole prefill (gitcode, sections "GDN prefill" and "API 全参数解析";
 * weigao.cc, "为什么要切成 64-token chunk"): the chunk-index build (large
 * batches only), the intra-chunk pass (gate log-cumsum, A, T), and the fused
 * pass that carries each state across chunks, writes checkpoints and the
 * final state (pool row state_indices[i] when given), and forms the output.
 * Runs gdn_validate_host() first and launches nothing when it fails.
 * Asynchronous on `stream`; returns GDN_OK once everything is enqueued, or
 * GDN_ERR_DEVICE (not a gfx950) / GDN_ERR_LAUNCH.  Data errors only the
 * device can see set bits in *status. */
int gdn_prefill(const gdn_prefill_params *p, void *stream);

/* gdn_prefill() with phase markers: events[i] (a hipEvent_t, or NULL to
 * skip) is recorded on `stream` just before phase i -- 0 chunk-index build,
 * 1 intra-chunk pass, 2 state pass, 3 output pass -- and events[4] after the
 * last, so hipEventElapsedTime(events[i], events[i + 1]) times phase i.  The
 * computation is exactly that of gdn_prefill().  events is a host array. */
int gdn_prefill_timed(const gdn_prefill_params *p, void *stream,
                      void *const events[5]);

/* gdn_prefill() for callers that cannot allocate device memory (code under
 * graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * workspace is a file-scope static device array of GDN_NOALLOC_SCRATCH_BYTES
 * (128 MiB) instead of p->workspace / p->workspace_bytes, which are ignored.
 * The caller still passes every input and output.  Nothing is allocated: no
 * hipMalloc, no hipFree, no allocating library call.  The first call on a
 * device looks up that device's copy of the array (hipGetSymbolAddress) and
 * keeps its address.  Returns GDN_ERR_SCRATCH when
 * gdn_prefill_workspace_size(p) exceeds GDN_NOALLOC_SCRATCH_BYTES (nothing
 * is launched), otherwise exactly what gdn_prefill() returns, with the same
 * results.  Every call on one GPU shares that GPU's array and leaves its
 * contents behind; no part of it needs to start at zero (every call writes
 * what it reads), but calls that overlap in time on one GPU (different
 * streams, or different host threads without ordering) race on it. */
int gdn_prefill_noalloc(const gdn_prefill_params *p, void *stream);

/*
 * One decode step: one new token per sequence, applied to the state with the
 * recurrence itself, no chunking (weigao.cc "GDN 与 Chunked Prefill", section
 * "Prefill 和 decode 的差异": after prefill each step adds a single token,
 * S <- alpha (I - beta k k^T) S + beta k v^T and o = scale * S^T q with the
 * updated S; gitcode "FlashInfer GDN Prefill 完全指南", sections "GDN
 * prefill" and "状态池": decode continues from the state prefill leaves, in
 * the same [rows, H, V, K] layout and state_indices pool).
 *
 * Takes the prefill parameter block with these differences:
 *   - token i is the new token of sequence i: total_tokens == num_seqs, and
 *     cu_seqlens must be NULL (GDN_ERR_SHAPE otherwise); q/k/v are
 *     [N, heads, D], g and beta [N, H], output [N, H, D];
 *   - checkpoint_every_n_tokens must be 0 and the checkpoint buffers NULL
 *     (GDN_ERR_CHECKPOINT); max_seqlen and the workspace are ignored;
 *   - q, k, v and output 16-byte aligned as in gdn_prefill (GDN_ERR_ALIGN);
 *     states whose rows are not 16-byte aligned are read and written element
 *     by element.
 * States, pools (output_state may alias initial_state), head sharing,
 * defaults, l2 normalisation and the status word behave as in gdn_prefill;
 * only GDN_STATUS_STATE_INDEX can be set.  Duplicate state_indices race.
 */
int gdn_decode(const gdn_prefill_params *p, void *stream);

/* The host-side checks of gdn_decode() alone; no GPU needed. */
int gdn_validate_decode_host(const gdn_prefill_params *p);

/*
 * The device-side chunk-index builder alone (weigao.cc, sections "chunked
 * prefill 有两层含义" and "为什么 trace 里它可能看起来很贵": the flat chunk ->
 * (sequence, chunk) table built on the device, with no device-to-host copy).
 *   cu_seqlens [N+1] (int32 or int64 per cu_type).
 *   chunk_indices [cap][2] int32: entry f = (sequence, chunk in sequence),
 *     sequence-major; entries at f >= n_chunks are (-1, -1).
 *     cap = gdn_max_chunks(total_tokens, num_seqs).
 *   cu_chunks [N+1] int32: exclusive prefix sum of ceil(len_i / 64).
 *   seq_starts [N+1] int32: the sequence starts actually used: cu_seqlens
 *     clamped into [0, T] and made non-decreasing (running maximum), so the
 *     table never exceeds cap even for invalid input (which also sets
 *     GDN_STATUS_CU_SEQLENS in *status).  Equal to cu_seqlens when it is
 *     valid.
 *   n_chunks [1] int32.  status: optional device word.
 * Every output buffer is caller-owned; cu_seqlens NULL means one sequence
 * [0, T] (num_seqs must then be 1).
 */
int gdn_build_chunk_indices(const void *cu_seqlens, int32_t cu_type,
                            int32_t num_seqs, int64_t total_tokens,
                            int32_t *chunk_indices, int32_t *cu_chunks,
                            int32_t *seq_starts, int32_t *n_chunks,
                            int32_t *status, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Gated linear recurrence: the diagonal sibling of the gated delta rule, over
 * the same packed sequences and state pools.  For every sequence and every
 * channel (h, d), with fp32 state,
 *
 *     h_t = g_t * h_{t-1} + x_t,      output_t = h_t
 *
 * from the given initial state (or zero).  g is the forget gate itself, in
 * [0, 1] (a gate above 1 is computed, but the products of 1 024 consecutive
 * gates of a sequence must stay finite).  An infinite state stays infinite under
 * gates above 0 and becomes NaN under a gate of 0, as the formula has it; states
 * that would leave fp32's range only halfway may become infinite.
 *
 * Shapes: x, output, doutput, dx [T, H, D] in x_dtype (F32, BF16 or F16); g,
 * dg [T, H, D], or [T, H] with g_per_head (one gate for the D channels of a
 * head; D must then be 32, 64 or 128), in g_dtype: F32 or x_dtype.  H and D
 * are any positive numbers with H * D < 2^29.  A call takes at most 2^30
 * sequences, ceil(T / 64) * ceil(H * D / 256) < 2^22 tiles and, in a decode
 * step, ceil(H * D / 4) * N <= 2^32 - 256 (GDN_ERR_SHAPE).  A token's H * D (or H) values are contiguous;
 * x, g and doutput have token strides in elements (0 = contiguous), every
 * other tensor is contiguous.  States are [rows, H, D] in any state dtype
 * with a row stride in elements (0 = contiguous); the 8-bit types saturate.
 * cu_seqlens, num_seqs, state_indices, pool_size and status are those of
 * gdn_prefill_params; output_state may be the same memory as initial_state,
 * and state_indices must be unique where a final state is written.  output may
 * be x itself (contiguous); no other two tensors of a call may overlap.
 * Tensors start on a boundary of their element size, the workspace on a
 * 256-byte boundary (GDN_ERR_ALIGN).  Calls that overlap in time need
 * workspaces of their own: if something else writes a call's workspace, the
 * call still ends and writes only its own buffers, but they hold NaN or other
 * wrong values.
 * Rows of output outside every sequence are untouched.  An empty sequence's
 * final state is its initial state.  A sequence whose state index is out of
 * range starts from zero and writes no final state.
 */
#define GDN_RECURRENCE_CHUNK 64 /* tokens per row of chunk_states */

typedef struct gdn_recurrence_params {
  int64_t total_tokens;    /* T >= 0 */
  int32_t num_seqs;        /* N >= 0; with cu_seqlens NULL, N must be 1 */
  int32_t num_heads;       /* H >= 1 */
  int32_t head_size;       /* D >= 1 */
  int32_t x_dtype;         /* gdn_dtype: F32, BF16, F16 */
  int32_t g_dtype;         /* F32 or x_dtype */
  int32_t g_per_head;      /* 0: g [T, H, D]; 1: g [T, H] */
  const void *x, *g;
  int64_t x_stride, g_stride;
  const void *cu_seqlens;  /* [N+1], NULL = one sequence [0, T] */
  int32_t cu_seqlens_type;
  void *output;
  const void *initial_state;
  int32_t initial_state_dtype;
  int64_t initial_state_stride;
  int32_t output_final_state;
  void *output_state;
  int32_t output_state_dtype;
  int64_t output_state_stride;
  const void *state_indices; /* [N] or NULL */
  int32_t state_indices_type;
  int64_t pool_size;
  /* fp32 [ceil(T / 64), H, D] or NULL.  gdn_recurrence() writes the state
   * before token 64 r into row r (rows whose first token starts a sequence or
   * lies outside every sequence hold unspecified values);
   * gdn_recurrence_backward() reads them, or forms them in its workspace at
   * the cost of one more pass over x and g when NULL. */
  float *chunk_states;
  /* gradients, gdn_recurrence_backward() only */
  const void *doutput;       /* [T, H, D] x_dtype */
  int64_t doutput_stride;
  const float *dfinal_state; /* [N, H, D] or NULL (zero) */
  void *dx, *dg;
  float *dinitial_state;     /* [N, H, D] or NULL (not formed) */
  void *workspace;
  size_t workspace_bytes;
  int32_t *status;           /* optional device word */
} gdn_recurrence_params;

/* Bytes of workspace gdn_recurrence() (backward == 0) or
 * gdn_recurrence_backward() (backward != 0) needs; only the shape fields and
 * whether chunk_states is given are read.  Host only; 0 can be a valid
 * answer: check the parameters with gdn_validate_recurrence_host(). */
size_t gdn_recurrence_workspace_size(const gdn_recurrence_params *p, int32_t backward);

/* The host-side checks of gdn_recurrence() (mode 0), its backward pass (1)
 * and its decode step (2); no GPU needed. */
int gdn_validate_recurrence_host(const gdn_recurrence_params *p, int32_t mode);

/* The forward pass: at most two kernels on `stream`. */
int gdn_recurrence(const gdn_recurrence_params *p, void *stream);

/* The backward pass, from x, g, the initial state, doutput (d loss / d
 * output) and dfinal_state (d loss / d final state):
 *   dh_t = doutput_t + g_{t+1} dh_{t+1}   (last token: + dfinal_state)
 *   dx_t = dh_t,  dg_t = dh_t h_{t-1}  (summed over D with g_per_head)
 *   dinitial_state = g_first dh_first     (empty sequence: dfinal_state)
 * The states are formed again in fp32 from x and g, so dg does not carry the
 * rounding of output.  dx and dg rows outside every sequence are zero.
 * state_indices must be NULL and output / output_state are ignored.  Results
 * do not depend on the order in which workgroups run. */
int gdn_recurrence_backward(const gdn_recurrence_params *p, void *stream);

/* One decode step: token i of x, g, output [N, ...] is the new token of
 * sequence i (total_tokens == num_seqs, cu_seqlens and chunk_states NULL).
 * No workspace. */
int gdn_recurrence_decode(const gdn_recurrence_params *p, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Rows of a state pool.  A pool is [rows, d1, d2, d3] of any state dtype with
 * four element strides (all zero = contiguous): the pools of gdn_prefill()
 * ([rows, H, V, K]) and of gdn_recurrence() ([rows, 1, H, D]).  At most
 * GDN_POOL_MAX_ROWS rows.  Row lists are device arrays (int32 or int64); an
 * entry of -1 is padding.  Entries outside the pool are skipped and set
 * GDN_STATUS_POOL_ROW.
 */
#define GDN_POOL_MAX_ROWS 262144

typedef struct gdn_pool_params {
  int64_t extent[3];        /* d1, d2, d3 >= 1 */
  const void *src;          /* gdn_pool_copy(); NULL otherwise */
  int32_t src_dtype;
  int64_t src_pool_rows;
  int64_t src_strides[4];
  void *dst;
  int32_t dst_dtype;
  int64_t dst_pool_rows;
  int64_t dst_strides[4];
  const void *src_rows;     /* [count] */
  const void *dst_rows;     /* [count] */
  int32_t rows_type;        /* gdn_itype of both lists */
  int64_t count;
  int32_t *status;          /* optional device word */
} gdn_pool_params;

/* The host-side checks of gdn_pool_copy() (mode 0), gdn_pool_reset() (1) and
 * gdn_pool_compact() (2). */
int gdn_validate_pool_host(const gdn_pool_params *p, int32_t mode);

/* dst[dst_rows[i]] = src[src_rows[i]] for every i: forking a row (one source,
 * several destinations), moving rows, or bringing rows of another pool or a
 * checkpoint buffer in, with conversion between state dtypes (to nearest; the
 * 8-bit types saturate; equal types copy bit for bit).  src and dst may be
 * the same view; other views may share no elements (GDN_ERR_STATE where they
 * do; and where their address ranges cross with different strides, so that the
 * host does not settle it).  A destination named twice takes its last
 * entry.  In one pool an entry whose source row is another entry's destination
 * is skipped, unless that one copies the row onto itself (it changes nothing, so
 * a row can be kept and forked in one list).  Both set their status bit.  At most GDN_POOL_MAX_ROWS entries
 * (GDN_ERR_SHAPE): each is compared with all others. */
int gdn_pool_copy(const gdn_pool_params *p, void *stream);

/* dst[dst_rows[i]] = 0 (rows freed, or taken for a new sequence). */
int gdn_pool_reset(const gdn_pool_params *p, void *stream);

/* Moves the live rows of dst to its front.  dst_rows [count] names the live
 * rows (a row may be named more than once).  With m distinct live rows, the
 * k-th live row at or behind row m (ascending) is copied to the k-th row
 * before m that is not live; new_rows [count] (same type, not overlapping
 * dst_rows) receives dst_rows with the moved rows renamed, invalid entries
 * as they are; num_live [1] (int32) receives m.  Rows at or behind m keep
 * their bytes, so the call can be repeated.  row_map [dst_pool_rows] (int32,
 * or NULL) receives each row's new place, -1 for rows that are not live. */
int gdn_pool_compact(const gdn_pool_params *p, void *new_rows, int32_t *num_live,
                     int32_t *row_map, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Short causal depthwise convolution of packed sequences, as layers put it in
 * front of a recurrence.  With x~ a sequence's state (its W - 1 last inputs from
 * before, zero without one) followed by its tokens,
 *
 *     output_t = act(bias + sum_j weight_j x~_{t + j}),  j < W, act: none or SiLU
 *
 * in fp32, rounded once; the final state is the last W - 1 rows of x~.
 *
 * Shapes: x, output, doutput, dx [T, C] in x_dtype (F32, BF16 or F16); weight
 * [C, W], bias [C] (or NULL) in weight_dtype: F32 or x_dtype; W is 2, 3 or 4.
 * x and doutput have token strides in elements (0 = contiguous); every other
 * tensor is contiguous.  States are [rows, W - 1, C], oldest row first, in any
 * state dtype with a row stride in elements (0 = contiguous).  cu_seqlens,
 * num_seqs, state_indices, pool_size and status are those of
 * gdn_prefill_params; output_state may be the same memory as initial_state,
 * and state_indices must be unique where a final state is written.  No other
 * two tensors of a call may overlap (GDN_ERR_STATE where output or dx meets x
 * or doutput); in a decode step output may be x itself, the same rows.  Tensors start on a
 * boundary of their element size.  Rows of output outside every sequence are
 * untouched, those of dx are zero.  A sequence whose state index is out of range
 * starts from zero and writes no final state.  A call takes at most 2^30
 * sequences and (ceil(T / 16) + N) * ceil(C / 64) < 2^26 (a decode step
 * ceil(C / 256) * N < 2^24; a backward pass also ceil((W + 1) C / 32) < 2^24);
 * GDN_ERR_SHAPE otherwise.
 */
typedef struct gdn_convolution_params {
  int64_t total_tokens;    /* T >= 0 */
  int32_t num_seqs;        /* N >= 0; with cu_seqlens NULL, N must be 1 */
  int32_t channels;        /* C >= 1 */
  int32_t width;           /* W: 2, 3 or 4 */
  int32_t x_dtype;         /* gdn_dtype: F32, BF16, F16 */
  int32_t weight_dtype;    /* F32 or x_dtype */
  int32_t silu;            /* 0: no activation, 1: SiLU */
  const void *x;
  int64_t x_stride;
  const void *weight, *bias;
  const void *cu_seqlens;  /* [N+1], NULL = one sequence [0, T] */
  int32_t cu_seqlens_type;
  void *output;
  const void *initial_state;
  int32_t initial_state_dtype;
  int64_t initial_state_stride;
  int32_t output_final_state;
  void *output_state;
  int32_t output_state_dtype;
  int64_t output_state_stride;
  const void *state_indices; /* [N] or NULL */
  int32_t state_indices_type;
  int64_t pool_size;
  /* gradients, gdn_convolution_backward() only */
  const void *doutput;       /* [T, C] x_dtype */
  int64_t doutput_stride;
  const float *dfinal_state; /* [N, W - 1, C] or NULL (zero) */
  void *dx;
  float *dweight;            /* [C, W] */
  float *dbias;              /* [C] or NULL (not formed) */
  float *dinitial_state;     /* [N, W - 1, C] or NULL (not formed) */
  void *workspace;
  size_t workspace_bytes;
  int32_t *status;           /* optional device word */
} gdn_convolution_params;

/* Bytes of workspace gdn_convolution() (backward == 0; more than 63 sequences
 * only) or gdn_convolution_backward() (backward != 0) needs.  Only the shape
 * fields are read.  Host only; 0 can be a valid answer. */
size_t gdn_convolution_workspace_size(const gdn_convolution_params *p, int32_t backward);

/* The host-side checks of gdn_convolution() (mode 0), its backward pass (1) and
 * its decode step (2); no GPU needed. */
int gdn_validate_convolution_host(const gdn_convolution_params *p, int32_t mode);

int gdn_convolution(const gdn_convolution_params *p, void *stream);

/* The backward pass.  state_indices must be NULL; output and output_state are
 * ignored.  Sums over tokens are formed in fp32 in a fixed order. */
int gdn_convolution_backward(const gdn_convolution_params *p, void *stream);

/* One decode step: token i of x, output [N, C] is the new token of sequence i
 * (total_tokens == num_seqs, cu_seqlens NULL).  No workspace. */
int gdn_convolution_decode(const gdn_convolution_params *p, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Selective state space scan of packed sequences.  With the step size
 * d_t = delta_t + delta_bias, or log(1 + e^ of it) with delta_softplus, for
 * every channel and each of its N states n, in fp32,
 *
 *     h_t = exp(d_t A) h_{t-1} + d_t B_t x_t
 *     y_t = sum_n C_t h_t + D x_t,     output_t = y_t, or y_t silu(z_t)
 *
 * from the given initial state (or zero).  A channel belongs to group
 * c / (channels / groups) of B and C.
 *
 * Shapes: x, delta, z (or NULL), output and their gradients [T, channels], B, C
 * and theirs [T, groups, N], all in x_dtype (F32, BF16 or F16); A [channels, N],
 * D, delta_bias [channels] (or NULL) fp32.  1 <= N <= 64.  x, delta, z, B, C and
 * doutput have token strides in elements (0 = contiguous); every other tensor is
 * contiguous.  States are [rows, channels, N] in any state dtype with a row
 * stride in elements (0 = contiguous).  cu_seqlens, num_seqs, state_indices,
 * pool_size and status are those of gdn_prefill_params; output_state may be the
 * same memory as initial_state, and state_indices must be unique where a final
 * state is written.  No other two tensors of a call may overlap (GDN_ERR_STATE
 * where output or a token's gradient meets x, delta, z, B, C or doutput).  Tensors
 * start on a boundary of their element size, the workspace on a 256-byte boundary.  Calls that overlap
 * in time need workspaces of their own.  Rows of output outside every sequence
 * are untouched, those of gradients are zero.  An empty sequence's final state
 * is its initial state.  A sequence whose state index is out of range starts
 * from zero and writes no final state.  The products exp(A sum d) over 256
 * consecutive tokens must stay finite (they do for A <= 0 and d >= 0).
 * An infinite state whose decay underflows fp32 within one token (d A below -87) is NaN
 * or infinite from there on.
 * channels <= 2^24, and T and the channels are limited by a grid's size (in a
 * decode step ceil(channels * ceil(N / 4) / 256) * num_seqs < 2^24, in a backward
 * pass ceil((N + 2) channels / 32) < 2^24);
 * GDN_ERR_SHAPE otherwise.
 */
typedef struct gdn_scan_params {
  int64_t total_tokens;    /* T >= 0 */
  int32_t num_seqs;        /* sequences; with cu_seqlens NULL, 1 */
  int32_t channels;
  int32_t num_states;      /* N */
  int32_t groups;          /* divides channels */
  int32_t x_dtype;         /* gdn_dtype: F32, BF16, F16 */
  int32_t delta_softplus;  /* 0 or 1 */
  const void *x, *delta, *z;
  int64_t x_stride, delta_stride, z_stride;
  const float *A;
  const void *B, *C;
  int64_t b_stride, c_stride;
  const float *D, *delta_bias;
  const void *cu_seqlens;  /* [num_seqs + 1], NULL = one sequence [0, T] */
  int32_t cu_seqlens_type;
  void *output;
  const void *initial_state;
  int32_t initial_state_dtype;
  int64_t initial_state_stride;
  int32_t output_final_state;
  void *output_state;
  int32_t output_state_dtype;
  int64_t output_state_stride;
  const void *state_indices; /* [num_seqs] or NULL */
  int32_t state_indices_type;
  int64_t pool_size;
  /* fp32 [ceil(T / gdn_scan_chunk()), N, channels] or NULL.  gdn_scan() writes
   * the states before every gdn_scan_chunk() tokens (what a row holds whose first
   * token no sequence reaches from before is not read); gdn_scan_backward() reads
   * them, or forms them in its workspace with one more pass when NULL. */
  float *chunk_states;
  /* gradients, gdn_scan_backward() only */
  const void *doutput;       /* [T, channels] x_dtype */
  int64_t doutput_stride;
  const float *dfinal_state; /* [num_seqs, channels, N] or NULL (zero) */
  void *dx, *ddelta, *dz;    /* dz: required with z */
  void *dB, *dC;
  float *dA;                 /* [channels, N] */
  float *dD, *ddelta_bias;   /* [channels] or NULL (not formed) */
  float *dinitial_state;     /* [num_seqs, channels, N] or NULL (not formed) */
  void *workspace;
  size_t workspace_bytes;
  int32_t *status;           /* optional device word */
} gdn_scan_params;

/* Tokens per row of chunk_states for these sizes (0: an invalid shape). */
int64_t gdn_scan_chunk(const gdn_scan_params *p);

/* Bytes of workspace gdn_scan() (backward == 0) or gdn_scan_backward() needs;
 * only the shape fields and whether chunk_states is given are read.  Which form a
 * forward pass takes depends on addresses too: the size is that of the form that needs
 * more, and a call may use little of it. */
size_t gdn_scan_workspace_size(const gdn_scan_params *p, int32_t backward);

/* The host-side checks of gdn_scan() (mode 0), its backward pass (1) and its
 * decode step (2); no GPU needed. */
int gdn_validate_scan_host(const gdn_scan_params *p, int32_t mode);

int gdn_scan(const gdn_scan_params *p, void *stream);

/* The backward pass.  state_indices must be NULL, initial_state fp32; output and
 * output_state are ignored.  The states are formed again in fp32.  Results do
 * not depend on the order in which workgroups run. */
int gdn_scan_backward(const gdn_scan_params *p, void *stream);

/* One decode step: token i of x, delta, z, B, C, output is the new token of
 * sequence i (total_tokens == num_seqs, cu_seqlens and chunk_states NULL).  No
 * workspace. */
int gdn_scan_decode(const gdn_scan_params *p, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Beam search: the best continuations of a group's beams.  Continuation v of
 * beam k scores scores_k + logits_kv - log sum_u exp(logits_ku); the
 * num_candidates best of a group's K V continuations are returned in descending
 * order, ties to the lowest beam, then the lowest token.  Sums over the
 * vocabulary are formed in fp32 (their parts joined in fp64), scores compared in
 * fp64 and returned in fp32.  A logit that is NaN or -inf, and every one of a
 * beam whose score is -inf or NaN (a beam that has ended), scores -inf; such
 * continuations come last, by beam and token.  Logits of +inf share the beam's
 * whole probability, and its other continuations score -inf.  Scores that are equal
 * in fp64 or infinite are ties, also those of unequal logits.
 */
#define GDN_BEAM_MAX 64 /* beams of a group, candidates of a group */

typedef struct gdn_beam_params {
  int32_t num_groups;      /* B >= 0 */
  int32_t num_beams;       /* K: 1 .. GDN_BEAM_MAX */
  int32_t vocab;           /* V: 1 .. 2^28 */
  int32_t num_candidates;  /* 1 .. GDN_BEAM_MAX, at most K V */
  int32_t logits_dtype;    /* F32, BF16 or F16 */
  const void *logits;      /* [B, K, V] */
  int64_t logits_stride;   /* elements from a beam to the next (0 = contiguous) */
  const float *scores;     /* [B, K] */
  float *out_scores;       /* [B, num_candidates] */
  int32_t *out_parents;    /* beams */
  int32_t *out_tokens;
  void *workspace;
  size_t workspace_bytes;
} gdn_beam_params;

size_t gdn_beam_workspace_size(const gdn_beam_params *p);
int gdn_validate_beam_host(const gdn_beam_params *p);
int gdn_beam_select(const gdn_beam_params *p, void *stream);

/* Brings the rows of state pools in the order of the selected parents.  Beam k
 * of group b holds row state_indices[b K + k] of every pool, rows all distinct;
 * child j of the group continues beam parents[b K + j].  The first child of a
 * parent keeps its row; the other children, in order, take the rows of the
 * beams without a child, in order, which are overwritten with their parents'
 * rows; no other row changes.  new_indices [B K] receives the children's rows.
 * An entry of parents outside [0, K) is no parent: its child takes a row that
 * is left over, as it is.  Rows outside the pool are handed on and neither read
 * nor written.  Both set GDN_STATUS_POOL_ROW (-1 does not: padding); a row that
 * is named twice sets GDN_STATUS_POOL_DUPLICATE, and what it holds afterwards is
 * unspecified.  Lists are int32 or int64, at most GDN_POOL_MAX_ROWS entries;
 * new_indices may not overlap them. */
typedef struct gdn_reorder_pool {
  void *pool;
  int32_t dtype;
  int64_t extent[3];   /* d1, d2, d3 >= 1, as in gdn_pool_params */
  int64_t strides[4];
} gdn_reorder_pool;

typedef struct gdn_reorder_params {
  int32_t num_groups;      /* B >= 0 */
  int32_t num_beams;       /* K: 1 .. GDN_BEAM_MAX */
  int32_t num_pools;       /* >= 1; GDN_ERR_STATE if two share elements */
  int64_t pool_rows;       /* rows of every pool */
  const gdn_reorder_pool *pools; /* host */
  const void *state_indices;
  const void *parents;
  void *new_indices;
  int32_t index_type;      /* gdn_itype of the three lists */
  int32_t *status;         /* optional device word */
} gdn_reorder_params;

int gdn_validate_reorder_host(const gdn_reorder_params *p);
int gdn_pool_reorder(const gdn_reorder_params *p, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_PREFILL_H */
