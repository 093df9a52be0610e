// The packed product with its epilogue, for one width of codes (linear.hip, compiled once for each).
#pragma once

#include "lowbit.h"
#include "moe.h"

namespace awq {

// Which kernel a call takes, and its grid; the same for all widths.
struct LinearPlan {
  bool tiles;        // linear_tile_kernel, else linear_rows_kernel or linear_few_kernel
  int blocks;        // row blocks of a tile: 16 rows each (few) or 32 (tiles)
  int waves;         // of a workgroup; few: they share the columns of K
  int64_t row_tiles;
  int col_tiles;
  int most;          // rows of a tile
  int team;          // > 0: linear_rows_kernel, so many of a workgroup's waves share a column tile
  int col_groups;    // its workgroups of a row tile
  size_t lds;        // and their LDS
};

template <int BITS>   // one for each of 2 to 8
hipError_t launch_linear_bits(const LinearArgs& a, awq_dtype_t dt, const LinearPlan& p, void* ws, hipStream_t st);

#define AWQ_LINEAR_DECLARE(b) \
  template <>                 \
  hipError_t launch_linear_bits<b>(const LinearArgs&, awq_dtype_t, const LinearPlan&, void*, hipStream_t)
AWQ_LINEAR_DECLARE(2);
AWQ_LINEAR_DECLARE(3);
AWQ_LINEAR_DECLARE(4);
AWQ_LINEAR_DECLARE(5);
AWQ_LINEAR_DECLARE(6);
AWQ_LINEAR_DECLARE(7);
AWQ_LINEAR_DECLARE(8);
#undef AWQ_LINEAR_DECLARE

}  // namespace awq
