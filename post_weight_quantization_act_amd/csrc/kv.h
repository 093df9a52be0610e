// What the rotary, cache and attention kernels share: argument blocks, the
// page lookups with their bounds, and the 8-bit code arithmetic.
#pragma once

#include "common.h"

namespace awq {

// A launch holds fewer than 2^32 threads: more make an error or, where the product wraps, a
// smaller grid.  `launch` gets the first workgroup and the number of each part of a grid.
template <class F>
void in_parts(int64_t blocks, int threads, F launch) {
  const int64_t most = ((1ll << 32) - 1) / threads / 64 * 64;   // the dealing over XCDs goes on as it was
  for (int64_t first = 0; first < blocks; first += most)
    launch((uint32_t)first, (unsigned)(blocks - first < most ? blocks - first : most));
}

// ---- rotary positions ---------------------------------------------------------
struct RopeFreqs {
  double base, factor, magnitude;
  double original, low, high;   // by parts: turns over `original` positions, kept / slowed outside [low, high]
  int kind;                     // awq_rope_scaling_kind_t
};

// f_i = base^(-2i/rot), slowed as `kind` says (fp64).
__host__ __device__ inline double rope_freq(const RopeFreqs& fr, int i, int half) {
  const double f = pow(fr.base, -(double)i / (double)half);
  if (fr.kind == AWQ_ROPE_SCALING_NONE) return f;
  if (fr.kind == AWQ_ROPE_SCALING_LINEAR) return f / fr.factor;
  const double turns = fr.original * f / 6.283185307179586476925;
  double w = fr.kind == AWQ_ROPE_SCALING_TURNS
                 ? (turns - fr.low) / (fr.high - fr.low)
                 : log(turns / fr.low) / log(fr.high / fr.low);
  w = w < 0.0 ? 0.0 : (w > 1.0 ? 1.0 : w);
  return w * f + (1.0 - w) * (f / fr.factor);
}

struct RopeArgs {
  const void* x;
  void* out;
  const int32_t* positions;   // may be null: the row's own index
  const float* table;
  int64_t B, S, H;
  int64_t xs[3], os[3];       // strides over B, S, H in elements
  int64_t pos_stride, n_pos;
  int D, rot, interleaved, transpose;
  uint32_t first_block;       // of the launch in its grid
};

// cos and sin of a position, NaN outside the table: a wrong position shows.
__device__ __forceinline__ float2 table_at(const float* table, int64_t n_pos, int half,
                                           int64_t pos, int i) {
  if (pos < 0 || pos >= n_pos) return make_float2(__builtin_nanf(""), __builtin_nanf(""));
  return ((const float2*)table)[pos * half + i];
}

// A product or sum that is rounded to fp32 before it is converted: without this the
// compiler may fold the operation and an fp16 conversion into one rounding.
__device__ __forceinline__ float fp32_value(float x) {
  asm("" : "+v"(x));
  return x;
}

__device__ __forceinline__ void rotate(float& x1, float& x2, float c, float s) {
  const float y1 = x1 * c - x2 * s;
  const float y2 = x2 * c + x1 * s;
  x1 = fp32_value(y1);
  x2 = fp32_value(y2);
}

// A unit is W pairs of a head in two runs of W columns (half layout: columns W u and
// rot/2 + W u; interleaved: 2 W u), or, past rot, columns that are not turned, where the
// second run may be missing.  W = 8 needs rot % 16 == 0, W = 4 rot % 8 == 0, both D % 8 == 0.
// Runs are read and written as vectors of any alignment.
struct Unit {
  int d0, d1;
  bool turn, two;
};

template <int W>
__host__ __device__ __forceinline__ int units_of(int D, int rot) {
  return rot / (2 * W) + (D - rot + 2 * W - 1) / (2 * W);
}

template <int W>
__device__ __forceinline__ Unit unit_of(int D, int rot, int interleaved, int u) {
  Unit r;
  r.turn = u < rot / (2 * W);
  if (r.turn) {
    r.d0 = interleaved ? 2 * W * u : W * u;
    r.d1 = interleaved ? 2 * W * u + W : rot / 2 + W * u;
    r.two = true;
  } else {
    r.d0 = 2 * W * u;
    r.d1 = 2 * W * u + W;
    r.two = r.d1 < D;
  }
  return r;
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x2 u32x2_loose __attribute__((aligned(2)));   // any element's address: the caller's strides
typedef u32x4 u32x4_loose __attribute__((aligned(2)));
typedef f32x4 f32x4_loose __attribute__((aligned(4)));

template <int W, class S> struct Run { S v[W]; };

template <int W, class S> __device__ __forceinline__ Run<W, S> load_run(const S* p) {
  if constexpr (sizeof(S) == 4) {
    struct { f32x4 v[W / 4]; } r;
#pragma unroll
    for (int i = 0; i < W / 4; ++i) r.v[i] = *(const f32x4_loose*)(p + 4 * i);
    return __builtin_bit_cast(Run<W, S>, r);
  } else if constexpr (W == 8) {
    return __builtin_bit_cast(Run<W, S>, *(const u32x4_loose*)p);
  } else {
    return __builtin_bit_cast(Run<W, S>, *(const u32x2_loose*)p);
  }
}
template <int W, class S> __device__ __forceinline__ void store_run(S* p, const float* x) {
  if constexpr (sizeof(S) == 4) {
#pragma unroll
    for (int i = 0; i < W; i += 4) *(f32x4_loose*)(p + i) = f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]};
  } else {
    Run<W, S> r;
#pragma unroll
    for (int i = 0; i < W; ++i) r.v[i] = from_f32<S>(x[i]);
    if constexpr (W == 8) *(u32x4_loose*)p = __builtin_bit_cast(u32x4, r);
    else *(u32x2_loose*)p = __builtin_bit_cast(u32x2, r);
  }
}
template <int W, class S> __device__ __forceinline__ void widen(const Run<W, S>& r, float* x) {
#pragma unroll
  for (int i = 0; i < W; ++i) x[i] = to_f32(r.v[i]);
}

// cos and sin of a unit's pairs.
template <int W>
struct Turns {
  float2 cs[W];
};
template <int W>
__device__ __forceinline__ Turns<W> turns_at(const float* table, int64_t n_pos, int half, int64_t pos,
                                             int u) {
  Turns<W> t;
  const bool in = pos >= 0 && pos < n_pos;
  const float* p = table + 2 * ((in ? pos : 0) * half + W * u);
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    const f32x4 v = *(const f32x4_loose*)(p + 4 * i);
    t.cs[2 * i] = make_float2(v[0], v[1]);
    t.cs[2 * i + 1] = make_float2(v[2], v[3]);
  }
  if (!in) {
#pragma unroll
    for (int i = 0; i < W; ++i) t.cs[i] = make_float2(__builtin_nanf(""), __builtin_nanf(""));
  }
  return t;
}

template <int W>
__device__ __forceinline__ void turn_unit(float* m0, float* m1, const Turns<W>& t, int interleaved,
                                          bool transpose) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float s = transpose ? -t.cs[i].y : t.cs[i].y;
    if (interleaved) {
      float* m = i < W / 2 ? m0 + 2 * i : m1 + 2 * (i - W / 2);
      rotate(m[0], m[1], t.cs[i].x, s);
    } else {
      rotate(m0[i], m1[i], t.cs[i].x, s);
    }
  }
}

// ---- the cache ------------------------------------------------------------------
struct KvArgs {
  uint8_t* k_codes;           // [n_pages][Hkv][P][D]
  uint8_t* v_codes;           // [n_pages][Hkv][D][P]
  float* k_steps;             // [n_pages][Hkv]
  float* v_steps;
  const int32_t* pages;       // [B][max_pages]
  const int32_t* starts;      // [B + 1] rows of each sequence; null: row b is sequence b's
  int64_t n_pages, T;
  int B, max_pages, Hkv, D, P, p_shift;
};

// Rows [row0, row0 + n) of sequence b, kept inside [0, T).
__device__ __forceinline__ void rows_of(const KvArgs& a, int b, int64_t& row0, int& n) {
  if (!a.starts) {
    row0 = b;
    n = b < a.T ? 1 : 0;
    return;
  }
  int64_t lo = a.starts[b], hi = a.starts[b + 1];
  lo = lo < 0 ? 0 : lo;
  hi = hi > a.T ? a.T : hi;
  row0 = lo;
  n = hi > lo ? (int)(hi - lo) : 0;
}

// Page id of a sequence's page p, or -1: outside the table or the pool there is none.
__device__ __forceinline__ int page_id(const KvArgs& a, int b, int64_t p) {
  if (p < 0 || p >= a.max_pages) return -1;
  const int id = a.pages[(int64_t)b * a.max_pages + p];
  return (unsigned)id < (uint64_t)a.n_pages ? id : -1;
}

// c = clamp(rint(q), -127, 127), 0 for NaN; stored as c + 128.
__device__ __forceinline__ int code_of(float q) {
  return q == q ? (int)__builtin_rintf(fminf(fmaxf(q, -127.0f), 127.0f)) : 0;
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

struct AppendArgs {
  KvArgs c;
  const void *k, *v, *q;
  void* q_out;
  const int32_t *lens, *positions;
  const float* table;
  int64_t ks[2], vs[2], qs[2];   // strides over rows and heads in elements
  int64_t n_pos;
  int rot, interleaved, Hq, pages_per_seq, max_new;
  int kv_blocks, q_parts;        // the launch's own
  awq_dtype_t q_type;            // of q_out
  uint32_t first_block;
};

struct ReadArgs {
  KvArgs c;
  const int32_t* first;
  void *k_out, *v_out;           // [T][Hkv][D]
  int pages_per_seq, max_new;
  uint32_t first_block;
};

struct AttArgs {
  KvArgs c;
  const void* q;
  void* out;                     // [T][Hq][D]
  float* lse;                    // [T][Hq] or null
  const int32_t* lens;
  int64_t qs[2];
  float scale;
  int Hq, causal, window, max_new, max_len;
  uint32_t first_block;
};

// Tokens [lo, hi) of the cache that row i of n of a sequence of `len` tokens sees; lo = hi:
// none.  Neither falls from a row to the next.
__device__ __forceinline__ void seen_by(const AttArgs& a, int len, int n, int i, int& lo, int& hi) {
  const int at = len - n + i;
  hi = a.causal ? at + 1 : len;
  lo = a.window > 0 && at >= a.window ? at - a.window + 1 : 0;   // at may be below 0: no overflow
  const int64_t table = (int64_t)a.c.max_pages << a.c.p_shift;   // past it there are no pages
  hi = hi > len ? len : hi;
  hi = hi > table ? (int)table : hi;
  hi = hi > a.max_len ? a.max_len : hi;
  hi = hi < 0 ? 0 : hi;
  lo = lo > hi ? hi : lo;   // a window that begins where no token is attended to any more
}

hipError_t launch_rope_table(int64_t n_pos, int rot, const RopeFreqs& fr, float* table,
                             hipStream_t st);
hipError_t launch_rope(const RopeArgs& a, awq_dtype_t in, awq_dtype_t out, hipStream_t st);
hipError_t launch_kv_append(const AppendArgs& a, awq_dtype_t in, hipStream_t st);
hipError_t launch_kv_read(ReadArgs a, awq_dtype_t out, hipStream_t st);
size_t kv_attention_ws_bytes(int64_t T, int64_t B, int Hq, int Hkv, int D, int max_new,
                             int max_len);   // of this call
size_t kv_attention_ws_bound(int64_t T, int64_t B, int Hq, int Hkv, int D, int max_new,
                             int max_len);   // of it and every smaller one
int64_t kv_attention_blocks(int64_t B, int Hq, int Hkv, int D, int max_new,
                            int max_len);   // workgroups of its largest grid
hipError_t launch_kv_attention(const AttArgs& a, awq_dtype_t dt, void* ws, hipStream_t st);

}  // namespace awq
