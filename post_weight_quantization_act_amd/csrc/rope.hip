// Rotary positions: the table of cosines and sines, and the rotation of
// strided [B, S, H, D] tensors (or its transpose, the gradient).
//
// Pair i < rot/2 of a head holds columns (i, i + rot/2) (half layout) or
// (2i, 2i + 1) (interleaved).  With c, s = table[position][i]:
//   y1 = x1 c - x2 s,   y2 = x2 c + x1 s          (transpose: s -> -s)
// in fp32, each product rounded and then the sum (the file is compiled without
// contraction), so that the appended codes agree bit for bit with any IEEE
// evaluation of these two lines.
#include "kv.h"

namespace awq {
namespace {

// Once for a model, in fp64, a pair a thread: 131072 positions of 64 pairs 84 us, 0.8 TB/s,
// bound by pow and sincos.
__global__ __launch_bounds__(256) void rope_table_kernel(int64_t n_pos, int half,
                                                         RopeFreqs fr, float2* table,
                                                         uint32_t first) {
  const int64_t e = ((int64_t)first + blockIdx.x) * 256 + threadIdx.x;
  if (e >= n_pos * half) return;
  const int64_t p = e / half;
  const int i = (int)(e % half);
  const double f = rope_freq(fr, i, half);
  double s, c;
  sincos((double)p * f, &s, &c);
  table[e] = make_float2((float)(c * fr.magnitude), (float)(s * fr.magnitude));
}

// rot % 8 == 0 and D % 8 == 0: a thread takes one unit (of eight pairs, or of four where
// rot % 16 is 8) of HB heads of a row, so that the row's
// cosines and sines are read once for them and HB heads' loads are in flight.  Bound by
// memory: 8191 rows x 64 heads x 128 columns, fp32 to bf16, 75 us, 5.4 TB/s (four heads;
// 79 us with one); the gradient of 8188 x 32 heads in fp16 28 us, 4.7 TB/s.  A pair a
// thread took 155 and 116 us.  Small calls take 3.2 us, one trip through memory and the
// launch.
template <class TI, class TO, int W, int HB>
__global__ __launch_bounds__(256) void rope_units_kernel(RopeArgs a, int rows_per_block) {
  typedef typename TI::storage SI;
  typedef typename TO::storage SO;
  const int units = units_of<W>(a.D, a.rot);
  const int blocks = (int)((a.H + HB - 1) / HB);
  const uint32_t work = (uint32_t)units * (uint32_t)blocks;     // threads' items of a row
  const uint32_t per_row = work < 256 ? work : 256;
  const uint32_t r = threadIdx.x / per_row;
  const int64_t row = ((int64_t)a.first_block + blockIdx.x) * rows_per_block + r;
  if ((int)r >= rows_per_block || row >= a.B * a.S) return;
  int64_t b, s;
  if ((uint64_t)(a.B * a.S) >> 32) {
    b = row / a.S;
    s = row % a.S;
  } else {
    b = (uint32_t)row / (uint32_t)a.S;
    s = (uint32_t)row % (uint32_t)a.S;
  }
  const SI* xr = (const SI*)a.x + b * a.xs[0] + s * a.xs[1];
  SO* yr = (SO*)a.out + b * a.os[0] + s * a.os[1];
  const int64_t pos = a.positions ? (int64_t)a.positions[b * a.pos_stride + s] : s;
  for (uint32_t e = threadIdx.x % per_row; e < work; e += per_row) {
    const int u = (int)(e % (uint32_t)units);
    const int64_t h0 = (int64_t)(e / (uint32_t)units) * HB;
    const Unit c = unit_of<W>(a.D, a.rot, a.interleaved, u);
    Run<W, SI> m0[HB], m1[HB];
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      const int64_t h = h0 + k < a.H ? h0 + k : h0;
      m0[k] = load_run<W>(xr + h * a.xs[2] + c.d0);
      m1[k] = load_run<W>(xr + h * a.xs[2] + (c.two ? c.d1 : c.d0));
    }
    Turns<W> t;
    if (c.turn) t = turns_at<W>(a.table, a.n_pos, a.rot >> 1, pos, u);
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      if (h0 + k >= a.H) break;
      float x0[W], x1[W];
      widen(m0[k], x0);
      widen(m1[k], x1);
      if (c.turn) turn_unit<W>(x0, x1, t, a.interleaved, a.transpose);
      SO* y = yr + (h0 + k) * a.os[2];
      store_run<W>(y + c.d0, x0);
      if (c.two) store_run<W>(y + c.d1, x1);
    }
  }
}

// Any rot and any row: one pair, or one column that is left as it is, a thread (the pairs
// of a rot that is no multiple of 8 do not fall into vectors).
template <class TI, class TO>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  typedef typename TI::storage SI;
  typedef typename TO::storage SO;
  const int half = a.rot >> 1;
  const int units = half + (a.D - a.rot);   // pairs, then the columns left as they are
  const int64_t e = ((int64_t)a.first_block + blockIdx.x) * 256 + threadIdx.x;
  if (e >= a.B * a.S * a.H * units) return;
  const int u = (int)(e % units);
  int64_t r = e / units;
  const int64_t h = r % a.H;
  r /= a.H;
  const int64_t s = r % a.S, b = r / a.S;
  const SI* x = (const SI*)a.x + b * a.xs[0] + s * a.xs[1] + h * a.xs[2];
  SO* y = (SO*)a.out + b * a.os[0] + s * a.os[1] + h * a.os[2];
  if (u >= half) {
    const int d = a.rot + (u - half);
    y[d] = from_f32<SO>(to_f32(x[d]));
    return;
  }
  const int64_t pos = a.positions ? (int64_t)a.positions[b * a.pos_stride + s] : s;
  const float2 cs = table_at(a.table, a.n_pos, half, pos, u);
  const int i1 = a.interleaved ? 2 * u : u, i2 = a.interleaved ? 2 * u + 1 : u + half;
  float x1 = to_f32(x[i1]), x2 = to_f32(x[i2]);
  rotate(x1, x2, cs.x, a.transpose ? -cs.y : cs.y);
  y[i1] = from_f32<SO>(x1);
  y[i2] = from_f32<SO>(x2);
}

template <class TI, class TO, int W, int HB>
void go_units(RopeArgs a, hipStream_t st) {
  const int64_t work = (int64_t)units_of<W>(a.D, a.rot) * ((a.H + HB - 1) / HB);
  const int rows = work < 256 ? (int)(256 / work) : 1;
  const int64_t blocks = (a.B * a.S + rows - 1) / rows;
  in_parts(blocks, 256, [&](uint32_t first, unsigned grid) {
    a.first_block = first;
    rope_units_kernel<TI, TO, W, HB><<<grid, 256, 0, st>>>(a, rows);
  });
}

template <class TI, class TO>
hipError_t go(RopeArgs a, hipStream_t st) {
  ProfScope prof("awq_rope", st);
  const bool rows = a.H * a.D <= 1ll << 34;    // a row's units are counted in 32 bits
  if (rows && a.rot % 16 == 0 && a.D % 8 == 0) {
    // four heads a thread for 2M units and more (4M units 74.9 against 79.0 us); one for fewer,
    // which need the threads (1M units of fp32 17.6 against 19.1 us)
    if (a.B * a.S * a.H * units_of<8>(a.D, a.rot) >= 2 << 20) go_units<TI, TO, 8, 4>(a, st);
    else go_units<TI, TO, 8, 1>(a, st);
  } else if (rows && a.rot % 8 == 0 && a.D % 8 == 0) {
    // 2 x 5066 rows x 64 heads x 80 columns of which 40 turn, bf16: 50 us (186 pair by pair)
    go_units<TI, TO, 4, 1>(a, st);
  } else {
    const int64_t n = a.B * a.S * a.H * (a.rot / 2 + a.D - a.rot);
    in_parts((n + 255) / 256, 256, [&](uint32_t first, unsigned grid) {
      a.first_block = first;
      rope_kernel<TI, TO><<<grid, 256, 0, st>>>(a);
    });
  }
  return hipGetLastError();
}

template <class TI>
hipError_t go_out(const RopeArgs& a, awq_dtype_t out, hipStream_t st) {
  if (out == AWQ_F32) return go<TI, F32T>(a, st);
  if (out == AWQ_F16) return go<TI, F16T>(a, st);
  return go<TI, BF16T>(a, st);
}

}  // namespace

hipError_t launch_rope_table(int64_t n_pos, int rot, const RopeFreqs& fr, float* table,
                             hipStream_t st) {
  const int64_t n = n_pos * (rot / 2);
  ProfScope prof("awq_rope_table", st);
  in_parts((n + 255) / 256, 256, [&](uint32_t first, unsigned grid) {
    rope_table_kernel<<<grid, 256, 0, st>>>(n_pos, rot / 2, fr, (float2*)table, first);
  });
  return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs& a, awq_dtype_t in, awq_dtype_t out, hipStream_t st) {
  if (in == AWQ_F32) return go_out<F32T>(a, out, st);
  if (in == AWQ_F16) return go_out<F16T>(a, out, st);
  return go_out<BF16T>(a, out, st);
}

}  // namespace awq
