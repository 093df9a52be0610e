// The paged key/value cache held in 8 bits: appending tokens (the keys rotated
// on the way, the queries with them) and reading token ranges back.
//
// A page holds P tokens of one sequence; each (page, head) block has one step
// for its keys and one for its values, the largest absolute value it has held
// divided by 127.  An append that raises a block's step moves the block's older
// codes to the new step, c' = rint(c * (step / step')).
// Compiled without contraction and with correctly rounded division: the codes
// agree bit for bit with any IEEE evaluation of these formulas.
#include "kv.h"

namespace awq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const uint32_t o = __shfl_xor(v, m);
    v = v > o ? v : o;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) v = v > red[w] ? v : red[w];
  return v;
}

template <class S>
__device__ __forceinline__ void load_pair(const AppendArgs& a, const S* x, int64_t pos, int u,
                                          int& i1, int& i2, float& x1, float& x2) {
  const int half = a.rot >> 1;
  i1 = a.interleaved ? 2 * u : u;
  i2 = a.interleaved ? 2 * u + 1 : u + half;
  x1 = to_f32(x[i1]);
  x2 = to_f32(x[i2]);
  const float2 cs = table_at(a.table, a.n_pos, half, pos, u);
  rotate(x1, x2, cs.x, cs.y);
}

template <class TI, class TQ>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a) {
  typedef typename TI::storage SI;
  typedef typename TQ::storage SQ;
  __shared__ uint32_t red[kThreads / 64];
  const KvArgs& c = a.c;
  int g = blockIdx.x;
  const int j = g % a.pages_per_seq;
  g /= a.pages_per_seq;
  const int h = g % c.Hkv, b = g / c.Hkv;
  int64_t row0;
  int n;
  rows_of(c, b, row0, n);
  const int64_t len = a.lens[b], first = len - n;   // places [first, len) are new
  const int64_t p = ((first < 0 ? 0 : first) >> c.p_shift) + j;
  const int64_t base = p << c.p_shift;
  if (n == 0 || base >= len) return;
  const int lo = (int)((first > base ? first : base) - base);       // first new place of the page
  const int hi = (int)((len < base + c.P ? len : base + c.P) - base);
  const int half = a.rot >> 1, units = half + (c.D - a.rot);
  const int64_t row_lo = row0 + (base + lo - first);
  const int tid = threadIdx.x;

  if (a.q) {   // this page's rows of the queries that share this head
    const int G = a.Hq / c.Hkv;
    const int work = (hi - lo) * G * units;
    for (int e = tid; e < work; e += kThreads) {
      const int u = e % units, r = e / units, hq = h * G + r % G;
      const int64_t row = row_lo + r / G;
      const SI* x = (const SI*)a.q + row * a.qs[0] + hq * a.qs[1];
      SQ* y = (SQ*)a.q_out + (row * a.Hq + hq) * c.D;
      if (u >= half) {
        const int d = a.rot + (u - half);
        y[d] = from_f32<SQ>(to_f32(x[d]));
        continue;
      }
      const int64_t pos = a.positions ? (int64_t)a.positions[row] : row - row0 + first;
      int i1, i2;
      float x1, x2;
      load_pair(a, x, pos, u, i1, i2, x1, x2);
      y[i1] = from_f32<SQ>(x1);
      y[i2] = from_f32<SQ>(x2);
    }
  }

  const int id = page_id(c, b, p);
  if (id < 0) return;   // no such page: its tokens are not kept
  const int64_t blk = (int64_t)id * c.Hkv + h;
  uint8_t* kc = c.k_codes + blk * c.P * c.D;
  uint8_t* vc = c.v_codes + blk * c.P * c.D;
  const bool old = lo > 0;
  const float k_was = old ? c.k_steps[blk] : 0.0f, v_was = old ? c.v_steps[blk] : 0.0f;

  uint32_t km = 0, vm = 0;
  for (int e = tid; e < (hi - lo) * units; e += kThreads) {
    const int u = e % units, r = e / units;
    const int64_t row = row_lo + r;
    const SI* x = (const SI*)a.k + row * a.ks[0] + h * a.ks[1];
    if (u >= half) {
      const uint32_t m = abs_bits(to_f32(x[a.rot + (u - half)]));
      km = km > m ? km : m;
      continue;
    }
    const int64_t pos = a.positions ? (int64_t)a.positions[row] : row - row0 + first;
    int i1, i2;
    float x1, x2;
    load_pair(a, x, pos, u, i1, i2, x1, x2);
    const uint32_t m1 = abs_bits(x1), m2 = abs_bits(x2);
    km = km > m1 ? km : m1;
    km = km > m2 ? km : m2;
  }
  for (int e = tid; e < (hi - lo) * c.D; e += kThreads) {
    const int d = e % c.D, r = e / c.D;
    const SI* x = (const SI*)a.v + (row_lo + r) * a.vs[0] + h * a.vs[1];
    const uint32_t m = abs_bits(to_f32(x[d]));
    vm = vm > m ? vm : m;
  }
  km = block_max(km, red);
  vm = block_max(vm, red);
  // a NaN's bits are above every number's, so a NaN among the values gives a NaN step
  const float kt = __uint_as_float(km) / 127.0f, vt = __uint_as_float(vm) / 127.0f;
  const float k_step = __float_as_uint(kt) > __float_as_uint(k_was) ? kt : k_was;
  const float v_step = __float_as_uint(vt) > __float_as_uint(v_was) ? vt : v_was;
  const bool k_grew = old && k_step != k_was, v_grew = old && v_step != v_was;

  // keys: older rows to the new step, then the new rows
  if (k_grew) {
    const float r = k_was / k_step;
    for (int e = tid; e < lo * c.D; e += kThreads)
      kc[e] = (uint8_t)(code_of((float)((int)kc[e] - 128) * r) + 128);
  }
  for (int e = tid; e < (hi - lo) * units; e += kThreads) {
    const int u = e % units, r = e / units;
    const int64_t row = row_lo + r;
    const SI* x = (const SI*)a.k + row * a.ks[0] + h * a.ks[1];
    uint8_t* y = kc + (int64_t)(lo + r) * c.D;
    if (u >= half) {
      const int d = a.rot + (u - half);
      y[d] = (uint8_t)((k_step > 0.0f ? code_of(to_f32(x[d]) / k_step) : 0) + 128);
      continue;
    }
    const int64_t pos = a.positions ? (int64_t)a.positions[row] : row - row0 + first;
    int i1, i2;
    float x1, x2;
    load_pair(a, x, pos, u, i1, i2, x1, x2);
    y[i1] = (uint8_t)((k_step > 0.0f ? code_of(x1 / k_step) : 0) + 128);
    y[i2] = (uint8_t)((k_step > 0.0f ? code_of(x2 / k_step) : 0) + 128);
  }
  // values: a row of the block is one column of the tokens
  for (int e = tid; e < c.D * hi; e += kThreads) {
    const int d = e % c.D, t = e / c.D;
    uint8_t* y = vc + (int64_t)d * c.P + t;
    if (t < lo) {
      if (v_grew) *y = (uint8_t)(code_of((float)((int)*y - 128) * (v_was / v_step)) + 128);
    } else {
      const SI* x = (const SI*)a.v + (row_lo + (t - lo)) * a.vs[0] + h * a.vs[1];
      *y = (uint8_t)((v_step > 0.0f ? code_of(to_f32(x[d]) / v_step) : 0) + 128);
    }
  }
  if (tid == 0) {
    c.k_steps[blk] = k_step;
    c.v_steps[blk] = v_step;
  }
}

template <class TO>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs a) {
  typedef typename TO::storage SO;
  const KvArgs& c = a.c;
  int g = blockIdx.x;
  const int j = g % a.pages_per_seq;
  g /= a.pages_per_seq;
  const int h = g % c.Hkv, b = g / c.Hkv;
  int64_t row0;
  int n;
  rows_of(c, b, row0, n);
  const int64_t first = a.first[b], end = first + n;
  const int64_t p = (first >> c.p_shift) + j, base = p << c.p_shift;
  if (n == 0 || base >= end) return;
  const int lo = (int)((first > base ? first : base) - base);
  const int hi = (int)((end < base + c.P ? end : base + c.P) - base);
  const int id = page_id(c, b, p);
  const int64_t blk = (int64_t)(id < 0 ? 0 : id) * c.Hkv + h;
  const uint8_t* kc = c.k_codes + blk * c.P * c.D;
  const uint8_t* vc = c.v_codes + blk * c.P * c.D;
  const float ks = c.k_steps[blk], vs = c.v_steps[blk];
  for (int e = threadIdx.x; e < (hi - lo) * c.D; e += kThreads) {
    const int d = e % c.D, t = lo + e / c.D;
    const int64_t o = ((row0 + (base + t - first)) * c.Hkv + h) * c.D + d;
    ((SO*)a.k_out)[o] = from_f32<SO>(id < 0 ? 0.0f : fp32_value((float)((int)kc[(int64_t)t * c.D + d] - 128) * ks));
    ((SO*)a.v_out)[o] = from_f32<SO>(id < 0 ? 0.0f : fp32_value((float)((int)vc[(int64_t)d * c.P + t] - 128) * vs));
  }
}

template <class TI>
hipError_t go_append(const AppendArgs& a, awq_dtype_t q_out, unsigned grid, hipStream_t st) {
  ProfScope prof("awq_kv_append", st);
  if (q_out == AWQ_F32) append_kernel<TI, F32T><<<grid, kThreads, 0, st>>>(a);
  else if (q_out == AWQ_F16) append_kernel<TI, F16T><<<grid, kThreads, 0, st>>>(a);
  else append_kernel<TI, BF16T><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, awq_dtype_t in, awq_dtype_t q_out,
                            hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)a.pages_per_seq * a.c.Hkv * a.c.B);
  if (in == AWQ_F32) return go_append<F32T>(a, q_out, grid, st);
  if (in == AWQ_F16) return go_append<F16T>(a, q_out, grid, st);
  return go_append<BF16T>(a, q_out, grid, st);
}

hipError_t launch_kv_read(const ReadArgs& a, awq_dtype_t out, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)a.pages_per_seq * a.c.Hkv * a.c.B);
  ProfScope prof("awq_kv_read", st);
  if (out == AWQ_F32) read_kernel<F32T><<<grid, kThreads, 0, st>>>(a);
  else if (out == AWQ_F16) read_kernel<F16T><<<grid, kThreads, 0, st>>>(a);
  else read_kernel<BF16T><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace awq
