// Internal declarations of the routed-FFN operators (experts.hip, grouped.hip,
// experts_api.hip).
#pragma once

#include "prox_internal.h"

namespace prox {

constexpr int kMaxExperts = 1024;  // experts of a router, groups of a product
constexpr int kMaxTopK = 32;
constexpr int kScaleBlock = 128;   // values that share one fp8 scale

// Whether a grid can be launched: blocks, and threads in all, have 32 bits.
inline bool grid_fits(int64_t blocks, int threads) {
  return blocks <= 0x7FFFFFFF && blocks * threads <= 0xFFFFFFFFll;
}

// Products of ragged groups of rows, out[r] = a[src(r)] W_g^T for the rows r of
// group g.  Strides are in bytes; every row of a and w starts 16-byte aligned
// and holds kbytes (a multiple of 16) bytes.
struct GroupedArgs {
  const uint8_t* a;
  const float* a_scale;      // [a_rows][kblocks], fp8 only
  const int* row_index;      // [rows] or nullptr: src(r) = r
  const int* offsets;        // [n_groups + 1] or nullptr: one group of all rows
  const uint8_t* w;          // [n_groups][n][k] (gated: up)
  const uint8_t* w_gate;     // gated products only
  const float* w_scale;      // [n_groups][nblocks][kblocks], fp8 only
  const float* w_gate_scale;
  uint8_t* out;
  int64_t a_stride, w_stride, w_group, out_stride;
  int a_rows, rows, n_groups, n, kbytes;
  int kblocks, nblocks;      // fp8 scale blocks of k and of n
  int wdtype, out_dtype, act;
};
hipError_t launch_grouped(const GroupedArgs& a, int cus, hipStream_t s);

struct RouteArgs {
  const void* logits;  // [tokens][experts]
  int logits_dtype, tokens, experts, top_k, renormalize;
  int* expert_idx;     // [tokens][top_k]
  float* weight;       // [tokens][top_k]
  int* offsets;        // [experts + 1]
  int* row_token;      // [tokens * top_k]
  int* row_of;         // [tokens][top_k]
  int* block_count;    // workspace: rows of each expert by block, int32 or bytes
};
size_t route_workspace(int tokens, int experts);  // bytes
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

struct QuantizeArgs {
  const uint8_t* x;
  uint8_t* q;
  float* scale;        // [ceil(rows / block_rows)][ceil(k / 128)]
  int64_t x_stride, q_stride;  // bytes
  int x_dtype, rows, k, block_rows;
};
hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t s);

struct CombineArgs {
  const uint8_t* h;
  const int* row_of;   // [tokens][top_k]
  const float* weight; // [tokens][top_k]
  uint8_t* y;
  int64_t h_stride, y_stride;  // bytes
  int h_dtype, y_dtype, h_rows, tokens, top_k, n;
  int vec;             // rows of h and y are 16-byte aligned and n is a multiple of 8
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t s);

// Error reporting shared with prox_api.hip (thread-local message).
prox_status fail(prox_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
prox_status hip_fail(hipError_t e, const char* what);
void clear_error();
int device_cus();

}  // namespace prox
