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

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest of two values over the workgroup (red: one pair for each wave).
template <bool WAVE = false>
__device__ __forceinline__ void block_max(uint32_t& k, uint32_t& v, uint2* red) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    k = umax(k, (uint32_t)__shfl_xor((int)k, m));
    v = umax(v, (uint32_t)__shfl_xor((int)v, m));
  }
  if (WAVE) return;
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = make_uint2(k, v);
  __syncthreads();
  for (int w = 0; w < waves; ++w) {
    k = umax(k, red[w].x);
    v = umax(v, red[w].y);
  }
}

// The step after the new tokens' largest value came in (bits of |x|: a NaN's are above
// every number's, so a NaN among the values gives a NaN step).
__device__ __forceinline__ float next_step(uint32_t top, float was) {
  const float step = __uint_as_float(top) / 127.0f;
  return __float_as_uint(step) > __float_as_uint(was) ? step : was;
}

__device__ __forceinline__ uint32_t coded(float x, float step) {
  return (uint32_t)((step > 0.0f ? code_of(x / step) : 0) + 128);
}

// The codes of a block's new values.  A step that is a number bounds the values by
// about 127 of it, so none is NaN and the quotient comes from the step's reciprocal
// (correctly rounded, five operations against eleven; both sides scaled by a power of
// two where the step is so small or large that a remainder would not be a normal
// number); a step of 0, or one that is not finite, makes every code 0, as the
// definition does.  Clamped, a quotient plus 2^23 + 128 is rounded to the nearest
// integer, ties to even, and its lowest byte is the stored code.
struct Coder {
  float step, inverse, scale;
  bool none;

  __device__ __forceinline__ explicit Coder(float s) {
    none = !(s > 0.0f && s < INFINITY);
    scale = s < 0x1p-60f ? 0x1p100f : s > 0x1p60f ? 0x1p-100f : 1.0f;
    step = s * scale;
    inverse = 1.0f / step;
  }
  __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) const {
    const uint32_t lo = __builtin_amdgcn_perm(bits(b), bits(a), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(bits(d), bits(c), 0x04000c0cu);
    return none ? 0x80808080u : lo | hi;
  }
  __device__ __forceinline__ uint32_t bits(float x) const {
    const float q = div_rn(x * scale, step, inverse);
    return __float_as_uint(__builtin_amdgcn_fmed3f(q, -127.0f, 127.0f) + 8388736.0f);
  }
};

// Codes of one dword to a step `by` times as coarse.
__device__ __forceinline__ uint32_t moved(uint32_t w, float by) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r |= (uint32_t)(code_of((float)((int)((w >> (8 * i)) & 255) - 128) * by) + 128) << (8 * i);
  return r;
}

// Where a workgroup of an append works: the new tokens [lo, hi) of a page of a sequence, of
// its first max_new rows (what the launch's registers are sized for).
struct Place {
  int64_t row_lo, row0, first;   // rows of token lo and of the sequence; number of its first new token
  int64_t page;                  // the sequence's page
  int lo, hi;
};

__device__ __forceinline__ bool find_place(const AppendArgs& a, int b, int j, Place& p) {
  const KvArgs& c = a.c;
  int n;
  rows_of(c, b, p.row0, n);
  const int64_t len = a.lens[b];
  p.first = len - n;
  p.page = ((p.first < 0 ? 0 : p.first) >> c.p_shift) + j;
  const int64_t base = p.page << c.p_shift, end = n < a.max_new ? len : p.first + a.max_new;
  if (n == 0 || base >= end) return false;
  p.lo = (int)((p.first > base ? p.first : base) - base);
  p.hi = (int)((end < base + c.P ? end : base + c.P) - base);
  p.row_lo = p.row0 + (base + p.lo - p.first);
  return true;
}

__device__ __forceinline__ int64_t position_of(const AppendArgs& a, const Place& p, int64_t row) {
  return a.positions ? (int64_t)a.positions[row] : row - p.row0 + p.first;
}

// Steps of a block before and after, and the factor for its older codes.
struct Steps {
  float k, v, k_by, v_by;
  bool k_grew, v_grew;
};

__device__ __forceinline__ Steps steps_after(const Place& p, float k_was, float v_was, uint32_t km,
                                             uint32_t vm) {
  Steps s;
  s.k = next_step(km, k_was);
  s.v = next_step(vm, v_was);
  s.k_grew = p.lo > 0 && s.k != k_was;
  s.v_grew = p.lo > 0 && s.v != v_was;
  s.k_by = k_was / s.k;
  s.v_by = v_was / s.v;
  return s;
}

// Turned queries leave in their own type (the same for a whole call).
template <int W>
__device__ __forceinline__ void store_query(const AppendArgs& a, int64_t at, const float* x) {
  if (a.q_type == AWQ_F16) store_run<W>((_Float16*)a.q_out + at, x);
  else if (a.q_type == AWQ_BF16) store_run<W>((__bf16*)a.q_out + at, x);
  else store_run<W>((float*)a.q_out + at, x);
}
__device__ __forceinline__ void store_query(const AppendArgs& a, int64_t at, float x) {
  if (a.q_type == AWQ_F16) ((_Float16*)a.q_out)[at] = from_f32<_Float16>(x);
  else if (a.q_type == AWQ_BF16) ((__bf16*)a.q_out)[at] = from_f32<__bf16>(x);
  else ((float*)a.q_out)[at] = x;
}

// rot % 8 == 0 (or no table).  A workgroup takes a page and head's keys and values, or
// (blocks from a.kv_blocks on) a part of the queries of a page's tokens.  The turned
// keys and the values stay in registers between the search for the largest and the
// rounding: HOLD units of 2 W keys, or patches of four tokens by four columns of
// values, a thread.
//
// Workgroups are dealt to the eight XCDs in turn: page number modulo 8 is the lowest
// digit, so the heads of a page, which turn by the same rows of the table, share an L2.
//
// 20005 tokens of 8 heads, 128 columns, pages of 64, bf16: 47 us with caches cold (123 MB
// of rows and codes and 10 MB of table, 2.8 TB/s), 37 warm; bound by the latency of load,
// largest, quotients, store in each workgroup, whose phases only other workgroups
// hide; with a division for each code 51 us, values' codes stored in the rows' order
// 51, one pair a thread 147.  One token of 192 sequences x 32 heads: 13.5 us, a chain
// of length, page, row and table loads; of one sequence 6.7 us.
template <class TI, int W, int HOLD>
__global__ __launch_bounds__(1024) void append_units_kernel(AppendArgs a) {
  typedef typename TI::storage SI;
  __shared__ uint2 red[16];
  const KvArgs& c = a.c;
  constexpr bool kWave = HOLD == 1;   // one token: a wave takes a head, a workgroup four
  const uint32_t block = a.first_block + blockIdx.x;
  const bool queries = block >= (uint32_t)a.kv_blocks;
  uint32_t g = queries ? block - a.kv_blocks : block;
  const uint32_t fan = queries ? a.q_parts : kWave ? (c.Hkv + 3) / 4 : c.Hkv, low = g & 7;
  g >>= 3;
  const int part = (int)(g % fan);
  const uint32_t at = g / fan * 8 + low;
  if (at >= (uint32_t)c.B * (uint32_t)a.pages_per_seq) return;
  const int j = (int)(at % (uint32_t)a.pages_per_seq), b = (int)(at / (uint32_t)a.pages_per_seq);
  Place p;
  if (!find_place(a, b, j, p)) return;
  const int units = units_of<W>(c.D, a.rot), tokens = p.hi - p.lo, half = a.rot >> 1;

  if (queries) {
    const int work = tokens * a.Hq * units, step = blockDim.x;
    for (int e = part * step + threadIdx.x; e < work; e += a.q_parts * step) {
      const int u = e % units, r = e / units, hq = r % a.Hq;
      const int64_t row = p.row_lo + r / a.Hq;
      const Unit w = unit_of<W>(c.D, a.rot, a.interleaved, u);
      const SI* x = (const SI*)a.q + row * a.qs[0] + hq * a.qs[1];
      float x0[W], x1[W];
      widen(load_run<W>(x + w.d0), x0);
      widen(load_run<W>(x + (w.two ? w.d1 : w.d0)), x1);
      if (w.turn)
        turn_unit<W>(x0, x1, turns_at<W>(a.table, a.n_pos, half, position_of(a, p, row), u),
                     a.interleaved, false);
      const int64_t y = (row * a.Hq + hq) * c.D;
      store_query<W>(a, y + w.d0, x0);
      if (w.two) store_query<W>(a, y + w.d1, x1);
    }
    return;
  }

  const int tid = kWave ? threadIdx.x & 63 : threadIdx.x, threads = kWave ? 64 : blockDim.x;
  const int h = kWave ? part * 4 + (threadIdx.x >> 6) : part;
  if (kWave && h >= c.Hkv) return;
  // the page's entry and steps, and the new rows: asked for together, looked at later
  const int id = page_id(c, b, p.page);
  const int64_t blk = (int64_t)(id < 0 ? 0 : id) * c.Hkv + h;

  // patches of values: tokens 4 t .. 4 t + 3 of the page, columns 4 d .. 4 d + 3, neighbours
  // along the tokens, so that a column's codes leave as one run
  const int t_lo = p.lo >> 2, t_n = ((p.hi + 3) >> 2) - t_lo, dq = c.D >> 2;
  const SI* v_rows = (const SI*)a.v + h * a.vs[1];
  SI v[HOLD][4][4];
  uint32_t vm = 0;
#pragma unroll
  for (int k = 0; k < HOLD; ++k) {
    const int e = tid + k * threads;
    if (e < t_n * dq) {
      const int d = e / t_n, t = 4 * (t_lo + e % t_n);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = t + i >= p.lo && t + i < p.hi;
        const SI* x = v_rows + (p.row_lo + (in ? t + i - p.lo : 0)) * a.vs[0] + 4 * d;
        const Run<4, SI> r = load_run<4>(x);
#pragma unroll
        for (int m = 0; m < 4; ++m) v[k][i][m] = in ? r.v[m] : (SI)0.0f;
      }
    }
  }
  float x0[HOLD][W], x1[HOLD][W];
  uint32_t km = 0;
  const SI* k_rows = (const SI*)a.k + h * a.ks[1];
#pragma unroll
  for (int k = 0; k < HOLD; ++k) {
    const int e = tid + k * threads;
    if (e < tokens * units) {
      const int u = e % units;
      const int64_t row = p.row_lo + e / units;
      const Unit w = unit_of<W>(c.D, a.rot, a.interleaved, u);
      const SI* x = k_rows + row * a.ks[0];
      widen(load_run<W>(x + w.d0), x0[k]);
      widen(load_run<W>(x + (w.two ? w.d1 : w.d0)), x1[k]);
      if (w.turn)
        turn_unit<W>(x0[k], x1[k], turns_at<W>(a.table, a.n_pos, half, position_of(a, p, row), u),
                     a.interleaved, false);
#pragma unroll
      for (int i = 0; i < W; ++i) km = umax(km, umax(abs_bits(x0[k][i]), abs_bits(x1[k][i])));
    }
  }
#pragma unroll
  for (int k = 0; k < HOLD; ++k)
    if (tid + k * threads < t_n * dq)
#pragma unroll
      for (int i = 0; i < 16; ++i) vm = umax(vm, abs_bits(to_f32(v[k][i >> 2][i & 3])));
  if (id < 0) return;   // no such page: its tokens are not kept
  const float k_was = p.lo > 0 ? c.k_steps[blk] : 0.0f, v_was = p.lo > 0 ? c.v_steps[blk] : 0.0f;
  block_max<kWave>(km, vm, red);
  const Steps s = steps_after(p, k_was, v_was, km, vm);
  const Coder key(s.k), value(s.v);

  uint8_t* kc = c.k_codes + blk * c.P * c.D;
  uint8_t* vc = c.v_codes + blk * c.P * c.D;
  if (s.k_grew) {
    uint32_t* w = (uint32_t*)kc;
    for (int e = tid; e < p.lo * dq; e += threads) w[e] = moved(w[e], s.k_by);
  }
#pragma unroll
  for (int k = 0; k < HOLD; ++k) {
    const int e = tid + k * threads;
    if (e < tokens * units) {
      const Unit w = unit_of<W>(c.D, a.rot, a.interleaved, e % units);
      uint8_t* y = kc + (p.lo + e / units) * c.D;
      const float *m = x0[k], *n = x1[k];
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        *(uint32_t*)(y + w.d0 + i) = key.four(m[i], m[i + 1], m[i + 2], m[i + 3]);
        if (w.two) *(uint32_t*)(y + w.d1 + i) = key.four(n[i], n[i + 1], n[i + 2], n[i + 3]);
      }
    }
  }
  // values: the dwords that hold older tokens, then the new ones over what of the last
  // such dword is theirs
  if (s.v_grew) {
    const int per = c.P >> 2, n = (p.lo + 3) >> 2;
    for (int e = tid; e < c.D * n; e += threads) {
      uint32_t* w = (uint32_t*)vc + (e / n) * per + e % n;
      *w = moved(*w, s.v_by);
    }
    __threadfence_block();
    if (!kWave) __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < HOLD; ++k) {
    const int e = tid + k * threads;
    if (e < t_n * dq) {
      const int d = e / t_n, t = 4 * (t_lo + e % t_n);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint8_t* y = vc + (4 * d + m) * c.P + t;
        const uint32_t r = value.four(to_f32(v[k][0][m]), to_f32(v[k][1][m]), to_f32(v[k][2][m]),
                                      to_f32(v[k][3][m]));
        if (t >= p.lo && t + 4 <= p.hi) {
          *(uint32_t*)y = r;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t + i >= p.lo && t + i < p.hi) y[i] = (uint8_t)(r >> (8 * i));
        }
      }
    }
  }
  if (tid == 0) {
    c.k_steps[blk] = s.k;
    c.v_steps[blk] = s.v;
  }
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

// Any rot, and prompts into pages of 256 tokens of more than 128 columns (more than a
// workgroup's registers hold): pairs one by one, the rows read twice (20005 tokens as above 147 us).
template <class TI>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a) {
  typedef typename TI::storage SI;
  __shared__ uint2 red[kThreads / 64];
  const KvArgs& c = a.c;
  int g = (int)(a.first_block + blockIdx.x);
  const int j = g % a.pages_per_seq;
  g /= a.pages_per_seq;
  const int h = g % c.Hkv, b = g / c.Hkv;
  Place p;
  if (!find_place(a, b, j, p)) return;
  const int lo = p.lo, hi = p.hi;
  const int64_t row_lo = p.row_lo;
  const int half = a.rot >> 1, units = half + (c.D - a.rot);
  const int tid = threadIdx.x;

  if (a.q) {   // this page's rows of the queries that share this head
    const int G = a.Hq / c.Hkv;
    const int work = (hi - lo) * G * units;
    for (int e = tid; e < work; e += kThreads) {
      const int u = e % units, r = e / units, hq = h * G + r % G;
      const int64_t row = row_lo + r / G;
      const SI* x = (const SI*)a.q + row * a.qs[0] + hq * a.qs[1];
      const int64_t y = (row * a.Hq + hq) * c.D;
      if (u >= half) {
        const int d = a.rot + (u - half);
        store_query(a, y + d, to_f32(x[d]));
        continue;
      }
      const int64_t pos = position_of(a, p, row);
      int i1, i2;
      float x1, x2;
      load_pair(a, x, pos, u, i1, i2, x1, x2);
      store_query(a, y + i1, x1);
      store_query(a, y + i2, x2);
    }
  }

  const int id = page_id(c, b, p.page);
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
      km = umax(km, abs_bits(to_f32(x[a.rot + (u - half)])));
      continue;
    }
    const int64_t pos = position_of(a, p, row);
    int i1, i2;
    float x1, x2;
    load_pair(a, x, pos, u, i1, i2, x1, x2);
    km = umax(km, umax(abs_bits(x1), abs_bits(x2)));
  }
  for (int e = tid; e < (hi - lo) * c.D; e += kThreads) {
    const int d = e % c.D, r = e / c.D;
    const SI* x = (const SI*)a.v + (row_lo + r) * a.vs[0] + h * a.vs[1];
    vm = umax(vm, abs_bits(to_f32(x[d])));
  }
  block_max(km, vm, red);
  const Steps s = steps_after(p, k_was, v_was, km, vm);

  // keys: older rows to the new step, then the new rows
  if (s.k_grew) {
    for (int e = tid; e < lo * c.D; e += kThreads)
      kc[e] = (uint8_t)(code_of((float)((int)kc[e] - 128) * s.k_by) + 128);
  }
  for (int e = tid; e < (hi - lo) * units; e += kThreads) {
    const int u = e % units, r = e / units;
    const int64_t row = row_lo + r;
    const SI* x = (const SI*)a.k + row * a.ks[0] + h * a.ks[1];
    uint8_t* y = kc + (int64_t)(lo + r) * c.D;
    if (u >= half) {
      const int d = a.rot + (u - half);
      y[d] = (uint8_t)coded(to_f32(x[d]), s.k);
      continue;
    }
    const int64_t pos = position_of(a, p, row);
    int i1, i2;
    float x1, x2;
    load_pair(a, x, pos, u, i1, i2, x1, x2);
    y[i1] = (uint8_t)coded(x1, s.k);
    y[i2] = (uint8_t)coded(x2, s.k);
  }
  // values: a row of the block is one column of the tokens
  for (int e = tid; e < c.D * hi; e += kThreads) {
    const int d = e % c.D, t = e / c.D;
    uint8_t* y = vc + (int64_t)d * c.P + t;
    if (t < lo) {
      if (s.v_grew) *y = (uint8_t)(code_of((float)((int)*y - 128) * s.v_by) + 128);
    } else {
      const SI* x = (const SI*)a.v + (row_lo + (t - lo)) * a.vs[0] + h * a.vs[1];
      *y = (uint8_t)coded(to_f32(x[d]), s.v);
    }
  }
  if (tid == 0) {
    c.k_steps[blk] = s.k;
    c.v_steps[blk] = s.v;
  }
}

// A thread takes four tokens by eight columns.  The values' four tokens are one
// dword of a column, so eight dwords and no transposition give four rows of
// eight; a workgroup runs over the heads of a page.  Bound by memory: 32760 tokens of
// 8 heads, 128 columns, to fp16 42 us, 4.8 TB/s, the rate of a copy (83 us with a value a
// thread).
template <class TO>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs a, int blocks) {
  typedef typename TO::storage SO;
  const KvArgs& c = a.c;
  uint32_t g = a.first_block + blockIdx.x;
  const int part = (int)(g % (uint32_t)blocks);
  g /= (uint32_t)blocks;
  const int j = (int)(g % (uint32_t)a.pages_per_seq), b = (int)(g / (uint32_t)a.pages_per_seq);
  int64_t row0;
  int n;
  rows_of(c, b, row0, n);
  const int64_t first = a.first[b], end = first + (n < a.max_new ? n : a.max_new);
  const int64_t p = (first >> c.p_shift) + j, base = p << c.p_shift;
  if (n == 0 || base >= end) return;
  const int lo = (int)((first > base ? first : base) - base);
  const int hi = (int)((end < base + c.P ? end : base + c.P) - base);
  const int d8 = c.D >> 3, t4 = c.P >> 2;
  const int e = part * kThreads + threadIdx.x;
  const int h = e / (d8 * t4);
  const int t = 4 * (e / d8 % t4), d = 8 * (e % d8);
  if (h >= c.Hkv || t >= hi || t + 4 <= lo) return;
  const int id = page_id(c, b, p);
  const int64_t blk = (int64_t)(id < 0 ? 0 : id) * c.Hkv + h;
  const uint8_t* kc = c.k_codes + (blk * c.P + t) * c.D + d;
  const uint8_t* vc = c.v_codes + (blk * c.D + d) * c.P + t;
  // a page that is not there reads as zero
  const float ks = id < 0 ? 0.0f : c.k_steps[blk], vs = id < 0 ? 0.0f : c.v_steps[blk];
  u32x2 k[4];
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) k[i] = *(const u32x2*)(kc + i * c.D);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = *(const uint32_t*)(vc + i * c.P);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (t + i < lo || t + i >= hi) continue;
    float x[8], y[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const uint32_t w = k[i][m >> 2];
      x[m] = fp32_value(((float)((w >> (8 * (m & 3))) & 255) - 128.0f) * ks);
      y[m] = fp32_value(((float)((v[m] >> (8 * i)) & 255) - 128.0f) * vs);
    }
    const int64_t o = ((row0 + (base + t + i - first)) * c.Hkv + h) * c.D + d;
    store_run<8>((SO*)a.k_out + o, x);
    store_run<8>((SO*)a.v_out + o, y);
  }
}

// Units of W pairs, if a workgroup's registers hold a page's.
template <class TI, int W>
bool go_units(AppendArgs a, hipStream_t st) {
  const int64_t pages = (int64_t)a.pages_per_seq * a.c.B;
  // as many threads as hold a page's new tokens: two units or patches each, four units of
  // four pairs where a page has more than 2 x 1024.  Four units of eight pairs and four
  // patches are more than the 128 registers that 1024 threads have each.
  const int64_t tokens = a.max_new < a.c.P ? a.max_new : a.c.P;
  const int64_t quads = (tokens + 6) / 4 < a.c.P / 4 ? (tokens + 6) / 4 : a.c.P / 4;
  const int64_t units = units_of<W>(a.c.D, a.rot);
  const int64_t k_items = tokens * units, v_items = quads * (a.c.D / 4);
  const int64_t items = k_items > v_items ? k_items : v_items;
  if (items > (W == 8 ? 2048 : 4096)) return false;
  const bool wave = items <= 64;       // one token, or a few of a narrow head
  const int threads = wave ? 256 : items > 2048 ? 1024 : (int)((items + 1) / 2 + 63) / 64 * 64;
  const int64_t eights = (pages + 7) / 8;
  a.kv_blocks = (int)(eights * (wave ? (a.c.Hkv + 3) / 4 : a.c.Hkv) * 8);
  a.q_parts = (int)((tokens * a.Hq * units + 4 * threads - 1) / (4 * threads));   // four units a thread
  if (a.q_parts > a.c.Hkv) a.q_parts = a.c.Hkv;
  in_parts(a.kv_blocks + eights * a.q_parts * 8, threads, [&](uint32_t first, unsigned grid) {
    a.first_block = first;
    if (wave) append_units_kernel<TI, W, 1><<<grid, threads, 0, st>>>(a);
    else if (W == 8 || items <= 2048) append_units_kernel<TI, W, 2><<<grid, threads, 0, st>>>(a);
    else append_units_kernel<TI, 4, 4><<<grid, threads, 0, st>>>(a);
  });
  return true;
}

template <class TI>
hipError_t go_append(AppendArgs a, hipStream_t st) {
  ProfScope prof("awq_kv_append", st);
  const bool done = a.rot % 16 == 0  ? go_units<TI, 8>(a, st)
                    : a.rot % 8 == 0 ? go_units<TI, 4>(a, st)
                                     : false;
  if (!done)
    in_parts((int64_t)a.pages_per_seq * a.c.Hkv * a.c.B, kThreads, [&](uint32_t first, unsigned grid) {
      a.first_block = first;
      append_kernel<TI><<<grid, kThreads, 0, st>>>(a);
    });
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, awq_dtype_t in, hipStream_t st) {
  if (in == AWQ_F32) return go_append<F32T>(a, st);
  if (in == AWQ_F16) return go_append<F16T>(a, st);
  return go_append<BF16T>(a, st);
}

hipError_t launch_kv_read(ReadArgs a, awq_dtype_t out, hipStream_t st) {
  const int blocks = (int)(((int64_t)a.c.Hkv * (a.c.P / 4) * (a.c.D / 8) + kThreads - 1) / kThreads);
  ProfScope prof("awq_kv_read", st);
  in_parts((int64_t)a.pages_per_seq * blocks * a.c.B, kThreads, [&](uint32_t first, unsigned grid) {
    a.first_block = first;
    if (out == AWQ_F32) read_kernel<F32T><<<grid, kThreads, 0, st>>>(a, blocks);
    else if (out == AWQ_F16) read_kernel<F16T><<<grid, kThreads, 0, st>>>(a, blocks);
    else read_kernel<BF16T><<<grid, kThreads, 0, st>>>(a, blocks);
  });
  return hipGetLastError();
}

}  // namespace awq
