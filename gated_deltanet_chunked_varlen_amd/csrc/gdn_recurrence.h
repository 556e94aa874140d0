// gdn_recurrence.h -- argument blocks and launchers of the gated linear
// recurrence and of the state-pool row operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gdn_prefill.h"

namespace gdn {

// GDN_OK if the current device is a gfx950; reports its CU count (gdn_host.hip).
int check_device(int *num_cus = nullptr);

// Tokens of one workgroup's tile in the backward scan, and in the forward scan
// by its types (eight times k6_recurrence.hip's tokens per wave).
constexpr int kRecTile = 64;
constexpr int rec_forward_tile(int x_dtype, int per_head) {
  return x_dtype != GDN_F32 && per_head ? 2 * kRecTile : kRecTile;
}
// Channels of one workgroup's tile: 64 lanes x 4.
constexpr int kRecChannels = 256;
// Tiles of one group of the chain, and the distance of two ticket counters
// (each in a cache line of its own).
constexpr int kGroup = 8;
constexpr int kTicketStep = 32;
__host__ __device__ constexpr int64_t groups_of(int64_t tiles) {
  return (tiles + kGroup - 1) / kGroup;
}

struct RecArgs {
  int64_t T;
  int32_t N, H, D, C;  // C = H * D channels
  int32_t x_dtype, g_dtype, g_per_head;
  const void *x, *g;
  int64_t x_stride, g_stride;  // elements per token
  void *out;
  const void *cu;
  int32_t cu_type;
  const int32_t *bos;  // sanitised sequence starts [N + 1]; NULL: N <= 63, from cu
  const void *init;    // states: element type and row stride
  int32_t init_dtype;
  int64_t init_stride;
  void *fin;
  int32_t fin_dtype;
  int64_t fin_stride;
  const void *sidx;
  int32_t sidx_type;
  int64_t pool_rows;
  float *chunk;  // [ceil(T / 64)][C] state before every 64 tokens, or NULL
  // backward
  const void *dy;
  int64_t dy_stride;
  const float *dfin;
  void *dx, *dg;
  float *dinit;
  // tiles and their chain
  int32_t ntiles, ncb;
  uint32_t units;             // ntiles * ncb
  int32_t empties;            // workgroups per channel block for the empty sequences
  uint32_t *ticket;           // [ncb][kTicketStep] next tile of a channel block; NULL: one tile
  unsigned long long *words;  // [ntiles][C], then
  unsigned long long *groups; // [ceil(ntiles / kGroup)][C]
  uint32_t wait_limit;        // looks at words that are not there before a wait gives up
  int32_t *status;
  int32_t vec;  // every row of x, g, dy, out, dx, dg is a whole number of aligned 4-element groups
  int32_t num_cus;
};

// wait_limit of a call: seconds, where a wait takes microseconds.  A variable for
// the sake of tests.
extern uint32_t rec_wait_limit;

int32_t rec_empties(uint32_t units, int32_t ncb, int32_t num_seqs);

// Clears the chain's words and ticket, and for N > 63 forms bos and the status.
hipError_t launch_rec_prepare(const RecArgs &a, int32_t *bos, hipStream_t s);
hipError_t launch_rec_forward(const RecArgs &a, hipStream_t s);
hipError_t launch_rec_backward(const RecArgs &a, hipStream_t s);
hipError_t launch_rec_decode(const RecArgs &a, hipStream_t s);

struct PoolArgs {
  int64_t row;  // elements of a row
  int64_t d2, d3;
  const void *src;
  int32_t src_dtype;
  int64_t src_pool;
  int64_t src_str[4];
  void *dst;
  int32_t dst_dtype;
  int64_t dst_pool;
  int64_t dst_str[4];
  const void *src_rows, *dst_rows;
  int32_t rows_type;
  int64_t count;
  int32_t *status;
  int32_t same;  // src and dst are one view
  // access: elements (or for equal types bytes) per thread and step, see k7_pool.hip
  int32_t flat;   // both rows contiguous
  int32_t align;  // largest power of two <= 16 that divides every row's address and length in bytes
  // compact
  void *new_rows;
  int32_t *num_live;
  int32_t *row_map;
  int32_t num_cus;
};

hipError_t launch_pool_copy(const PoolArgs &a, hipStream_t s);
hipError_t launch_pool_reset(const PoolArgs &a, hipStream_t s);
hipError_t launch_pool_compact(const PoolArgs &a, hipStream_t s);

}  // namespace gdn
