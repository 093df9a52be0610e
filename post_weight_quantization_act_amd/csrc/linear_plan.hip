// Which kernel a packed product takes, and with how many workgroups.
#include <algorithm>

#include "linear.h"

namespace awq {
namespace {

LinearPlan plan(const LinearArgs& a) {
  LinearPlan p;
  const int outputs = a.gated ? a.N / 2 : a.N;
  // rows that an expert has if all have alike
  const int64_t each = a.offsets ? (a.rows + a.experts - 1) / a.experts : a.rows;
  p.tiles = each > 64;
  int64_t most;
  if (p.tiles) {
    p.waves = 4;
    p.blocks = 4;
    most = 32 * p.blocks;
    p.col_tiles = (outputs + (a.gated ? 127 : 255)) / (a.gated ? 128 : 256);
  } else {
    p.blocks = each <= 16 ? 1 : each <= 32 ? 2 : 4;
    p.waves = p.blocks == 4 ? 4 : 8;
    most = 16 * p.blocks;
    p.col_tiles = (outputs + (a.gated ? 15 : 31)) / (a.gated ? 16 : 32);
  }
  // each expert may leave a part of a tile, and so may the rows that none has
  p.row_tiles = a.offsets ? std::min(a.rows, a.rows / most + a.experts + 1) : (a.rows + most - 1) / most;
  return p;
}

}  // namespace

size_t linear_ws_bytes(const LinearArgs&, awq_dtype_t) { return 0; }

int64_t linear_threads(const LinearArgs& a) {
  const LinearPlan p = plan(a);
  return p.row_tiles * p.col_tiles * 64 * p.waves;
}

hipError_t launch_linear(const LinearArgs& a, awq_dtype_t dt, int bits, void* ws, hipStream_t st) {
  const LinearPlan p = plan(a);
  switch (bits) {
    case 2: return launch_linear_bits<2>(a, dt, p, ws, st);
    case 3: return launch_linear_bits<3>(a, dt, p, ws, st);
    case 4: return launch_linear_bits<4>(a, dt, p, ws, st);
    case 5: return launch_linear_bits<5>(a, dt, p, ws, st);
    case 6: return launch_linear_bits<6>(a, dt, p, ws, st);
    case 7: return launch_linear_bits<7>(a, dt, p, ws, st);
    default: return launch_linear_bits<8>(a, dt, p, ws, st);
  }
}

}  // namespace awq
