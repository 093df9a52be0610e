// The packed product with its epilogue, for one width of codes (linear.hip, compiled once for each).
#pragma once

#include "kv.h"
#include "lowbit.h"
#include "moe.h"

namespace awq {

// Rows that are taken from bf16 to fp16 have their largest element at 2^kRowScale and up to twice that.
constexpr int kRowScale = 15;

// ---- epilogue ------------------------------------------------------------------------------
// exp, quotients and tanh from the hardware's exp2 and reciprocal (an ulp each): relative error
// a few 2^-24 and that of the exponent's own rounding, |v| 2^-24, which v's rounding to fp32, |v| 2^-24 of it too,
// makes of the result in any form.  tanh's form is v / (1 + exp(-2 u)).
__device__ __forceinline__ float over_one_plus_exp(float v, float minus) {
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(minus * -1.44269504088896341f));
}
template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == AWQ_ACT_RELU) return v < 0.0f ? 0.0f : v;
  else if constexpr (ACT == AWQ_ACT_SILU) return over_one_plus_exp(v, v);
  else if constexpr (ACT == AWQ_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  else if constexpr (ACT == AWQ_ACT_GELU_TANH)
    return over_one_plus_exp(v, 1.5957691216057307f * fmaf(0.044715f * v, v * v, v));
  else return v;
}

__device__ __forceinline__ float load_as(const void* p, int64_t i, int type) {
  if (type == AWQ_F32) return ((const float*)p)[i];
  return type == AWQ_F16 ? (float)((const _Float16*)p)[i] : (float)((const __bf16*)p)[i];
}
__device__ __forceinline__ void store_as(void* p, int64_t i, int type, float v) {
  if (type == AWQ_F32) ((float*)p)[i] = v;
  else if (type == AWQ_F16) ((_Float16*)p)[i] = (_Float16)v;
  else ((__bf16*)p)[i] = (__bf16)v;
}

// N outputs of a row from column n on, from their sums, gates and ups where gated.
template <int ACT, int N>
__device__ __forceinline__ void finish_act(const LinearArgs& a, int expert, int64_t row, int n, float (&v)[N],
                                           float (&up)[N]) {
  const int outputs = a.gated ? a.N / 2 : a.N;
  if (a.bias) {
    const float* b = a.bias + (int64_t)expert * a.N + n;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] += b[i];
      if (a.gated) up[i] += b[outputs + i];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = activate<ACT>(v[i]);
    if (a.gated) v[i] *= up[i];
  }
  if (a.residual) {
    const int64_t at = row * a.residual_stride + n;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += load_as(a.residual, at + i, a.out_type);
  }
  const int64_t at = row * outputs + n;
  if constexpr (N == 1) {
    store_as(a.out, at, a.out_type, v[0]);
  } else if (a.out_type == AWQ_F32) {
    store_run<N>((float*)a.out + at, v);
  } else if (a.out_type == AWQ_F16) {
    store_run<N>((_Float16*)a.out + at, v);
  } else {
    store_run<N>((__bf16*)a.out + at, v);
  }
}
template <int N>
__device__ __forceinline__ void finish(const LinearArgs& a, int expert, int64_t row, int n, float (&v)[N], float (&up)[N]) {
  switch (a.act) {
    case AWQ_ACT_RELU: return finish_act<AWQ_ACT_RELU>(a, expert, row, n, v, up);
    case AWQ_ACT_SILU: return finish_act<AWQ_ACT_SILU>(a, expert, row, n, v, up);
    case AWQ_ACT_GELU: return finish_act<AWQ_ACT_GELU>(a, expert, row, n, v, up);
    case AWQ_ACT_GELU_TANH: return finish_act<AWQ_ACT_GELU_TANH>(a, expert, row, n, v, up);
    default: return finish_act<AWQ_ACT_NONE>(a, expert, row, n, v, up);
  }
}

// Which kernel a call takes, and its grid; the same for all widths.
struct LinearPlan {
  bool tiles;        // linear_tile_kernel, else linear_few_kernel
  int blocks;        // row blocks of a tile: 16 rows each (few) or 32 (tiles)
  int waves;         // of a workgroup; few: they share the columns of K
  int64_t row_tiles;
  int col_tiles;
  int splits, per;   // tiles: parts of K with a workgroup each, and their steps of 128 columns
  float* partial;    // splits > 1: the parts' sums [splits][rows][N]
};

template <int BITS>   // one for each of 2 to 8
hipError_t launch_linear_bits(const LinearArgs& a, awq_dtype_t dt, const LinearPlan& p, hipStream_t st);

#define AWQ_LINEAR_DECLARE(b) \
  template <>                 \
  hipError_t launch_linear_bits<b>(const LinearArgs&, awq_dtype_t, const LinearPlan&, hipStream_t)
AWQ_LINEAR_DECLARE(2);
AWQ_LINEAR_DECLARE(3);
AWQ_LINEAR_DECLARE(4);
AWQ_LINEAR_DECLARE(5);
AWQ_LINEAR_DECLARE(6);
AWQ_LINEAR_DECLARE(7);
AWQ_LINEAR_DECLARE(8);
#undef AWQ_LINEAR_DECLARE

}  // namespace awq
