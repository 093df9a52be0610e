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

__global__ __launch_bounds__(256) void rope_table_kernel(int64_t n_pos, int half,
                                                         RopeFreqs fr, float2* table) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= n_pos * half) return;
  const int64_t p = e / half;
  const int i = (int)(e % half);
  const double f = rope_freq(fr, i, half);
  double s, c;
  sincos((double)p * f, &s, &c);
  table[e] = make_float2((float)(c * fr.magnitude), (float)(s * fr.magnitude));
}

template <class TI, class TO>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  typedef typename TI::storage SI;
  typedef typename TO::storage SO;
  const int half = a.rot >> 1;
  const int units = half + (a.D - a.rot);   // pairs, then the columns left as they are
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
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

template <class TI, class TO>
hipError_t go(const RopeArgs& a, hipStream_t st) {
  const int64_t n = a.B * a.S * a.H * (a.rot / 2 + a.D - a.rot);
  ProfScope prof("awq_rope", st);
  rope_kernel<TI, TO><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a);
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
  rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(n_pos, rot / 2, fr,
                                                                 (float2*)table);
  return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs& a, awq_dtype_t in, awq_dtype_t out, hipStream_t st) {
  if (in == AWQ_F32) return go_out<F32T>(a, out, st);
  if (in == AWQ_F16) return go_out<F16T>(a, out, st);
  return go_out<BF16T>(a, out, st);
}

}  // namespace awq
