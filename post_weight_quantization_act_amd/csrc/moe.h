// What the kernels around a block of experts share: argument blocks, and how sorted rows
// are found.
#pragma once

#include "common.h"

namespace awq {

constexpr int kMostExperts = 1024;
constexpr int kMostChosen = 32;

// Pairs (token, choice) sorted by expert.  Bucket e < count holds expert first + e's, bucket
// `count` those of experts elsewhere.
struct SortArgs {
  const int32_t* experts;        // [n]
  int32_t *offsets, *order, *place;
  int32_t* hist;                 // [blocks][count + 1]: how many pairs of a block a bucket has
  int64_t n;
  int64_t per;                   // pairs of a block
  int blocks, first, count;
};

struct RouteArgs {
  SortArgs s;                    // offsets may be null: nothing is sorted
  const void* logits;
  const float* bias;
  int32_t* experts;
  float* weights;
  int64_t T, stride;
  float scale;
  int E, k, sigmoid, normalise;
};

struct RouteGradArgs {
  const void* logits;
  const int32_t* experts;
  const float* dweights;
  void* dlogits;                 // [T][E]
  int64_t T, stride;
  float scale;
  int E, k, sigmoid, normalise;
  uint32_t first_block;
};

// Tokens [T][C] against sorted rows [T k][C].
struct RowsArgs {
  const void *tokens, *rows;     // what is read; either may be null
  void* out;                     // tokens or sorted rows
  const float* weights;          // [T][k]; null: 1
  float* dots;                   // [T][k], or null
  const int32_t *offsets, *place;
  int64_t T, C, stride;          // row stride of `tokens`
  int k, count;
  uint32_t first_block;
};

size_t moe_sort_ws_bytes(int64_t n, int count);
hipError_t launch_moe_sort(SortArgs a, hipStream_t st);
hipError_t launch_moe_route(RouteArgs a, awq_dtype_t dt, hipStream_t st);
hipError_t launch_moe_route_grad(RouteGradArgs a, awq_dtype_t dt, hipStream_t st);
hipError_t launch_moe_gather(RowsArgs a, awq_dtype_t dt, hipStream_t st);
// out [T][C] of out_dt = tokens (or 0) + sum of weighted rows
hipError_t launch_moe_combine(RowsArgs a, awq_dtype_t dt, awq_dtype_t out_dt, hipStream_t st);
// out (sorted rows of dt, may be null) = weighted tokens of token_dt; dots = tokens . rows of dt
hipError_t launch_moe_combine_grad(RowsArgs a, awq_dtype_t token_dt, awq_dtype_t dt, hipStream_t st);

// linear.hip
struct LinearArgs {
  const void* x;
  const uint32_t* codes;         // [K/32][experts N][bits]
  const float2* meta;            // [K/group][experts N]
  const float* bias;             // [experts][N] or null
  const void* residual;          // [rows][outputs] of the output's type, or null
  void* out;                     // [rows][outputs]
  const int32_t *offsets, *order;   // null: all rows are expert 0's; rows as they are
  const float* x_scale;          // [x_rows]: what a row of x is to be multiplied by; null: 1
  int64_t K, stride, residual_stride, x_rows;
  int64_t R;                     // rows of all experts' weights
  int64_t rows;
  int N, experts, per_token, lg_cpg, act, gated, out_type;
  bool grouped;                  // offsets are given
};
// from rows, x_rows, N, K, experts, gated, grouped: of this call, and of it and every one with fewer rows
size_t linear_ws_bytes(const LinearArgs& a, awq_dtype_t dt);
size_t linear_ws_bound(LinearArgs a, awq_dtype_t dt);
int64_t linear_threads(const LinearArgs& a);   // of the call's grid
hipError_t launch_linear(LinearArgs a, awq_dtype_t dt, int bits, void* ws, hipStream_t st);

}  // namespace awq
