// Which kernel a packed product takes, and with how many workgroups.
#include <algorithm>

#include "linear.h"

namespace awq {
namespace {

// bf16 rows as fp16 ones: scaled by the power of two that takes their largest finite element to
// [2^15, 2^16), the last one that fp16 has, they keep all bits down to 2^-32 of it, and further down an error
// of at most 2^-40 of it: 2^-16 of the rounding of a sum that has it.  A wave a row; scale is the
// factor that is left beside kRowScale's.
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
      top = m < 0x7f80u && m > top ? m : top;
    }
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const uint32_t o = __shfl_xor(top, m);
    top = top > o ? top : o;
  }
  int e = (int)(top >> 7) - 127;
  e = top == 0 ? 0 : e < -126 ? -126 : e;
  for (int64_t k = 8 * lane; k < K; k += 512) {
    const bf16x8 v = *(const bf16x8*)(p + k);
    half8 y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (_Float16)ldexpf((float)v[i], kRowScale - e);
    *(half8*)(out + row * K + k) = y;
  }
  if (lane == 0) scale[row] = ldexpf(1.0f, e);
}

// Whether bf16 activations of a large call are taken to fp16 first: unpacking takes half the
// instructions then, 2 to 4% of a call, and the pass as many bytes again as x has.  From 4096
// products for each element on (4095 tokens, 6 of 64 experts, 2816 x 2048, 4 bits: 353 us without,
// 344 with; the same rows, sorted, 2048 x 1408: no gain).  They are dense then, and stay within a
// buffer's 4 GiB where overlapping ones would not; the pass's grid stays below 2^32 threads at 32 columns.
constexpr int64_t kMostScaled = (1ll << 31) - 129;
bool scaled(const LinearArgs& a, awq_dtype_t dt, const LinearPlan& p) {
  return dt == AWQ_BF16 && p.tiles && p.blocks == 4 && a.rows * a.N >= 4096 * a.x_rows && a.x_rows * a.K <= kMostScaled;
}

// The parts' sums [splits][rows][N], added in their order, and the rest of the product.  Bound by memory,
// the caches' for the most part: 64 rows of 4096 columns in 8 parts are 8 MB.
__global__ __launch_bounds__(256) void join_kernel(LinearArgs a, LinearPlan p, uint32_t runs) {
  const uint32_t at = blockIdx.x * 256 + threadIdx.x;
  const int64_t row = at / runs;
  if (row >= a.rows) return;
  const int outputs = a.gated ? a.N / 2 : a.N, n = 4 * (int)(at % runs);
  const float* from = p.partial + row * a.N + n;
  const int64_t apart = a.rows * a.N;
  if (n + 4 <= outputs) {
    float v[4] = {}, up[4] = {};
    for (int s = 0; s < p.splits; ++s) {
      const Run<4, float> x = load_run<4>(from + s * apart);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += x.v[i];
      if (a.gated) {
        const Run<4, float> y = load_run<4>(from + s * apart + outputs);
#pragma unroll
        for (int i = 0; i < 4; ++i) up[i] += y.v[i];
      }
    }
    finish(a, 0, row, n, v, up);
  } else {
    for (int i = 0; n + i < outputs; ++i) {
      float v[1] = {0.0f}, up[1] = {0.0f};
      for (int s = 0; s < p.splits; ++s) {
        v[0] += from[s * apart + i];
        if (a.gated) up[0] += from[s * apart + outputs + i];
      }
      finish(a, 0, row, n + i, v, up);
    }
  }
}

// All times are of a call with 4-bit codes in groups of 128 and bf16 rows.
LinearPlan plan(const LinearArgs& a) {
  LinearPlan p = {};
  const int outputs = a.gated ? a.N / 2 : a.N, steps = (int)((a.K + 127) / 128);
  const int cols = (outputs + (a.gated ? 127 : 255)) / (a.gated ? 128 : 256);     // column tiles
  auto parts = [&](int64_t most) { return (a.rows + most - 1) / most; };
  // rows that an expert has if all have alike, and experts that have any
  const int64_t each = a.grouped ? parts(a.experts) : a.rows, busy = a.grouped ? std::min<int64_t>(a.rows, a.experts) : 1;
  // Few rows: 16 rows of 4096 x 11008 20 us, 32 in tiles; 32 rows of 11008 x 4096 27 and 28, of 28672 x
  // 4096 51 and 32.  64 experts, 2816 x 2048: 32 rows 31 and 34, 64 rows 50 and 37.  8 experts, 32 rows
  // each, of 512 x 2048: 15 and 29.
  const bool few = a.grouped ? a.rows < a.experts || (each <= 32 && busy * cols < 128)
                             : a.rows <= 16 || (a.rows <= 32 && cols <= 48);
  p.splits = 1;
  if (few) {
    p.blocks = each <= 16 ? 1 : 2;
    p.col_tiles = (outputs + (a.gated ? 15 : 31)) / (a.gated ? 16 : 32);
    // as many waves as run at once: 1 x 28672 x 8192 38 us with 8 waves, 36 with 4, 45 with 2; 1 x 4096 x
    // 11008 17, 26 and 45
    p.waves = busy * p.col_tiles >= 512 ? 4 : 8;
  } else {
    p.tiles = true;
    p.col_tiles = cols;
    // 64 experts, 2816 x 2048, as many rows for each, with 1, 2 and 4 blocks of 32 rows: 32 rows each 73, 70
    // and 103 us (drawn alike, with 1 block 69, and 55 for 32 each), 16 rows
    // 58, 64 and 96, 80 rows 138, 127 and 141, 256 rows 315, 268 and 276; 384 rows of 2048 x 1408 223
    // with 2 and 214 with 4.  One projection: 256 rows of 28672 x 4096 106, 89 and 84 us, 2048 rows of
    // 4096 x 11008 283, 229 and 206.
    auto groups = [&]() { return a.grouped ? busy * ((each + 32 * p.blocks - 1) / (32 * p.blocks)) * cols : parts(32 * p.blocks) * cols; };
    if (a.grouped) {
      p.blocks = each <= 32 ? 1 : each <= 256 ? 2 : 4;
      // smaller tiles where there is not one for each compute unit: 8 experts, 128 rows each, of 512 x
      // 2048: 39 us with 2 blocks, 30 with 1
      while (p.blocks > 1 && groups() < 256) p.blocks /= 2;
    } else {
      p.blocks = parts(128) * cols >= 256 ? 4 : a.rows <= 64 ? 1 : 2;
    }
    // where tiles leave compute units idle, K in parts of at least four steps: 64 rows of 4096 x 11008
    // 92 us without, 33 with 8 parts of K; 512 rows 129 and 78
    if (!a.grouped && p.blocks < 4)
      while (2 * p.splits * groups() <= 512 && steps >= 8 * p.splits) p.splits *= 2;
    p.per = (steps + p.splits - 1) / p.splits;
    p.splits = (steps + p.per - 1) / p.per;
    // two sets of waves where a workgroup has a compute unit to itself, for smaller tiles half of them: 8
    // experts, 64 rows each, of 512 x 2048 (32 tiles) 29 us with one set and 24 with two, 16 rows of
    // 8192 x 2048 (256) 32 and 32, 24 rows 40 and 47
    p.waves = groups() * p.splits <= (p.blocks == 4 ? 256 : 128) ? 8 : 4;
  }
  // each expert may leave a part of a tile, and so may the rows that none has
  const int most = (p.tiles ? 32 : 16) * p.blocks;
  p.row_tiles = a.grouped ? std::min(a.rows, a.rows / most + a.experts + 1) : parts(most);
  return p;
}

}  // namespace

size_t linear_ws_bytes(const LinearArgs& a, awq_dtype_t dt) {
  const LinearPlan p = plan(a);
  return scaled(a, dt, p) ? (size_t)a.x_rows * (a.K * 2 + 4) : p.splits > 1 ? (size_t)p.splits * a.rows * a.N * 4 : 0;
}

// Parts of K: their number changes where the row tiles do, at multiples of 32 rows, and between two of those
// what they need grows with the rows; from 256 tiles on, so at 16384 rows at the latest, there are none. Scaled
// rows: tiles of 128 rows once there stay with more rows, so the largest call that has them has all of a.rows.
size_t linear_ws_bound(LinearArgs a, awq_dtype_t dt) {
  const LinearPlan p = plan(a);
  size_t most = linear_ws_bytes(a, dt);
  if (dt == AWQ_BF16 && p.tiles && p.blocks == 4) {
    const int64_t x_rows = std::min({a.x_rows, a.rows * a.N / 4096, kMostScaled / a.K});
    most = std::max(most, (size_t)x_rows * (a.K * 2 + 4));
  }
  if (a.grouped) return most;
  const int64_t rows = a.rows;
  for (a.rows = 32; a.rows < rows && a.rows <= 16384; a.rows += 32) {
    const LinearPlan q = plan(a);
    if (q.splits > 1) most = std::max(most, (size_t)q.splits * a.rows * a.N * 4);
  }
  return most;
}

int64_t linear_threads(const LinearArgs& a) {
  const LinearPlan p = plan(a);
  return p.row_tiles * p.col_tiles * 64 * p.waves * p.splits;
}

hipError_t launch_linear(LinearArgs a, awq_dtype_t dt, int bits, void* ws, hipStream_t st) {
  LinearPlan p = plan(a);
  p.partial = (float*)ws;
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
  const hipError_t e = [&] {
    switch (bits) {
      case 2: return launch_linear_bits<2>(a, dt, p, st);
      case 3: return launch_linear_bits<3>(a, dt, p, st);
      case 4: return launch_linear_bits<4>(a, dt, p, st);
      case 5: return launch_linear_bits<5>(a, dt, p, st);
      case 6: return launch_linear_bits<6>(a, dt, p, st);
      case 7: return launch_linear_bits<7>(a, dt, p, st);
      default: return launch_linear_bits<8>(a, dt, p, st);
    }
  }();
  if (e != hipSuccess || p.splits == 1) return e;
  const int outputs = a.gated ? a.N / 2 : a.N, runs = (outputs + 3) / 4;
  ProfScope prof("awq_lowbit_linear_join", st);
  join_kernel<<<(unsigned)((a.rows * runs + 255) / 256), 256, 0, st>>>(a, p, (uint32_t)runs);
  return hipGetLastError();
}

}  // namespace awq
