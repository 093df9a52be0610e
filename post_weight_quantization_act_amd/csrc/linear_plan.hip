// Which kernel a packed product takes, and with how many workgroups.
#include <algorithm>

#include "linear.h"

namespace awq {
namespace {

// bf16 rows as fp16 ones: scaled by the power of two that takes their largest below 2, they keep all
// bits down to 2^-16 of it, and 24 bits below that largest further down.  A row that is not finite
// is left unscaled.  A wave a row.
__global__ __launch_bounds__(256) void scale_rows_kernel(const __bf16* x, int64_t rows, int64_t K, int64_t stride,
                                                         _Float16* out, float* scale) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const __bf16* p = x + row * stride;
  uint32_t top = 0;
  for (int64_t k = 8 * lane; k < K; k += 512) {
    const u16x8 v = *(const u16x8*)(p + k);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = v[i] & 0x7fffu;
      top = top > m ? top : m;
    }
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const uint32_t o = __shfl_xor(top, m);
    top = top > o ? top : o;
  }
  int e = (int)(top >> 7) - 127;
  e = top == 0 || top >= 0x7f80u ? 0 : e < -126 ? -126 : e;
  for (int64_t k = 8 * lane; k < K; k += 512) {
    const bf16x8 v = *(const bf16x8*)(p + k);
    half8 y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (_Float16)ldexpf((float)v[i], -e);
    *(half8*)(out + row * K + k) = y;
  }
  if (lane == 0) scale[row] = ldexpf(1.0f, e);
}

// Whether bf16 activations of a tile kernel's call are taken to fp16 first: unpacking takes half the
// instructions then, 2 to 4% of a call, and the pass as many bytes again as x has.  From 4096
// products for each element on (4095 tokens, 6 of 64 experts, 2816 x 2048, 4 bits: 353 us without,
// 344 with; the same rows, sorted, 2048 x 1408: no gain).
bool scaled(const LinearArgs& a, awq_dtype_t dt, const LinearPlan& p) {
  return dt == AWQ_BF16 && p.tiles && a.rows * a.N >= 4096 * a.x_rows;
}

LinearPlan plan(const LinearArgs& a) {
  LinearPlan p = {};
  const int outputs = a.gated ? a.N / 2 : a.N;
  // rows that an expert has if all have alike
  const int64_t each = a.offsets ? (a.rows + a.experts - 1) / a.experts : a.rows;
  // each expert may leave a part of a tile, and so may the rows that none has
  auto tiles = [&](int most) {
    p.most = most;
    p.row_tiles = a.offsets ? std::min(a.rows, a.rows / most + a.experts + 1) : (a.rows + most - 1) / most;
  };
  p.tiles = each > 64;
  if (p.tiles) {
    p.blocks = 4;
    p.col_tiles = (outputs + (a.gated ? 127 : 255)) / (a.gated ? 128 : 256);
    tiles(128);
    p.waves = (a.rows + 127) / 128 * p.col_tiles <= 256 ? 8 : 4;
    return p;
  }
  p.col_tiles = (outputs + (a.gated ? 15 : 31)) / (a.gated ? 16 : 32);
  if (each <= 32) {
    // experts differ: room for twice the rows, so that most have one tile
    const int64_t room = std::min(a.rows, a.offsets ? 2 * each : each);
    const int most = room <= 16 ? (int)room : 32;
    p.blocks = most == 32 ? 2 : 1;
    p.lds = (size_t)most * (a.K + 8) * 2 + 32 * 1024 * p.blocks;   // and the waves' sums
    if (p.lds <= 150 * 1024) {
      tiles(most);
      p.waves = 8;
      // as many waves as run at once
      const int64_t busy = a.offsets ? std::min<int64_t>(a.rows, a.experts) : p.row_tiles, work = busy * p.col_tiles;
      p.team = work >= 4096 ? 1 : work >= 2048 ? 2 : work >= 1024 ? 4 : 8;
      const int64_t wide = 8 / p.team, per = std::max<int64_t>(1, (work / wide + 511) / 512);
      p.col_groups = (int)((p.col_tiles + wide * per - 1) / (wide * per));
      return p;
    }
  }
  p.blocks = each <= 16 ? 1 : each <= 32 ? 2 : 4;
  p.waves = p.blocks == 4 ? 4 : 8;
  tiles(16 * p.blocks);
  return p;
}

}  // namespace

size_t linear_ws_bytes(const LinearArgs& a, awq_dtype_t dt) {
  return scaled(a, dt, plan(a)) ? (size_t)a.x_rows * (a.K * 2 + 4) : 0;
}

int64_t linear_threads(const LinearArgs& a) {
  const LinearPlan p = plan(a);
  return p.row_tiles * p.col_tiles * 64 * p.waves;     // and fewer where a workgroup takes several columns
}

hipError_t launch_linear(LinearArgs a, awq_dtype_t dt, int bits, void* ws, hipStream_t st) {
  const LinearPlan p = plan(a);
  if (scaled(a, dt, p)) {
    _Float16* x = (_Float16*)ws;
    float* scale = (float*)(x + a.x_rows * a.K);
    {
      ProfScope prof("awq_lowbit_linear_scale", st);
      scale_rows_kernel<<<(unsigned)((a.x_rows + 3) / 4), 256, 0, st>>>((const __bf16*)a.x, a.x_rows, a.K, a.stride, x, scale);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.x = x;
    a.stride = a.K;
    a.x_scale = scale;
    dt = AWQ_F16;
  }
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
