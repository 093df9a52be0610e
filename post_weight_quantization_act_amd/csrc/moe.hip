// Around a block of experts: the router, tokens sorted by expert, rows there and back.
//
// Pair t k + j is token t's j-th choice.  Sorted rows are the pairs by expert, an expert's
// in their own order, and last, past offsets[count], pairs of experts elsewhere.
#include <algorithm>
#include <type_traits>

#include "kv.h"
#include "moe.h"

namespace awq {
namespace {

// ---- over the 16 lanes of a row -----------------------------------------------------
template <int N>
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  return __builtin_amdgcn_update_dpp(0, x, 0x120 + N, 0xf, 0xf, false);
}
template <int N>
__device__ __forceinline__ double turned(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  return __longlong_as_double((long long)((uint64_t)turned<N>((uint32_t)(u >> 32)) << 32 | turned<N>((uint32_t)u)));
}
template <class F>
__device__ __forceinline__ uint32_t row_all(uint32_t x, F f) {
  x = f(x, turned<8>(x));
  x = f(x, turned<4>(x));
  x = f(x, turned<2>(x));
  return f(x, turned<1>(x));
}
__device__ __forceinline__ uint32_t row_umax(uint32_t x) {
  return row_all(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint32_t row_umin(uint32_t x) {
  return row_all(x, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
__device__ __forceinline__ uint32_t row_or(uint32_t x) {
  return row_all(x, [](uint32_t a, uint32_t b) { return a | b; });
}
__device__ __forceinline__ float row_max(float x) {
  return __uint_as_float(row_all(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float row_sum(float x) {
  return __uint_as_float(row_all(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ double row_sum(double x) {
  x += turned<8>(x);
  x += turned<4>(x);
  x += turned<2>(x);
  return x + turned<1>(x);
}
__device__ __forceinline__ uint64_t row_umax(uint64_t x) {
  const uint32_t hi = row_umax((uint32_t)(x >> 32));
  const uint32_t lo = row_umax((uint32_t)(x >> 32) == hi ? (uint32_t)x : 0u);
  return (uint64_t)hi << 32 | lo;
}

// ---- the router -------------------------------------------------------------------------
// Keys that order as the scores do: 0 for what is taken or not there, 1 for NaN, which ranks last.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 1u;
  const uint32_t u = __float_as_uint(x + 0.0f);    // -0 and 0 are equal
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double x) {
  if (x != x) return 1ull;
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// The `count` largest keys of 16 lanes' VPL each, the lowest number of equals: f(j, key, number) for
// the j-th.  Keys that are taken become 0.
template <int VPL, class Key, class F>
__device__ __forceinline__ void take_largest(Key (&key)[VPL], int l, int count, F f) {
  for (int j = 0; j < count; ++j) {
    Key best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool more = key[i] > best;
      best = more ? key[i] : best;
      at = more ? i : at;
    }
    const Key top = row_umax(best);
    const uint32_t won = row_umin(best == top ? (uint32_t)(l + 16 * at) : 0xffffffffu);
    f(j, top, (int)won);
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = won == (uint32_t)(l + 16 * i) ? (Key)0 : key[i];
  }
}

// The sigmoids p of the chosen logits v (choice j in lane j % 16 of a row) and, normalise, over their sum.
// In 32 bits one below 2^-126 loses bits and one below e^-88 is 0, and so is the sum where all are: a row
// with a logit below -80 is taken in 64, which are whole down to -708 and 0 below -745.  16381 x 256 with a
// bias as before, 22 us.
__device__ __forceinline__ void sigmoids(const float (&v)[2], const bool (&there)[2], bool normalise, float by, float (&p)[2]) {
  constexpr float kLow = -80.0f;
  float f[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) f[s] = there[s] ? 1.0f / (1.0f + expf(-v[s])) : 0.0f;
  const float sum = normalise ? row_sum(f[0] + f[1]) : 1.0f;
#pragma unroll
  for (int s = 0; s < 2; ++s) p[s] = sum == 0.0f ? 0.0f : f[s] / sum * by;
  const bool low = row_or((there[0] && v[0] < kLow) || (there[1] && v[1] < kLow)) != 0;
  if (!__any(low)) return;
  double d[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) d[s] = there[s] ? 1.0 / (1.0 + exp(-(double)v[s])) : 0.0;
  const double total = normalise ? row_sum(d[0] + d[1]) : 1.0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const float exact = total == 0.0 ? 0.0f : (float)(d[s] / total * by);
    p[s] = low ? exact : p[s];
  }
}

__device__ __forceinline__ float value_of(uint32_t key) {
  return key <= 1u ? __builtin_nanf("") : __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key);
}

// One token by 16 lanes, lane l holding the logits l, l + 16, ..  Choice j ends in lane j % 16.
// Without a bias the scores order as the logits.  With one they are defined in 64 bits.  They are
// formed in 32 first, within 4 2^-24 + 2^-24 |score| of that (sigmoid: exp2, a sum, a reciprocal, the
// bias); where two neighbours among the chosen and the next lie closer than four times as much, once in
// some thousand tokens, the choice is made again in 64 bits: 16381 tokens of 256 logits take 21 to 25
// us, and 35 to 41 in 64 bits alone.
template <class S, int VPL, bool BIAS>
__device__ __forceinline__ void route_token(const RouteArgs& a, const S* row, int l, int (&index)[2],
                                            float (&weight)[2]) {
  float x[VPL];
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int c = l + 16 * i;
    x[i] = c < a.E ? to_f32(row[c]) : -INFINITY;
  }
  index[0] = index[1] = 0;
  auto keep = [&](int j, int won) __attribute__((always_inline)) {
    if (l == (j & 15)) {
      if (j < 16) index[0] = won;
      else index[1] = won;
    }
  };
  if constexpr (!BIAS) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = l + 16 * i < a.E ? key_of(x[i]) : 0u;
    take_largest<VPL>(key, l, a.k, [&](int j, uint32_t, int won) __attribute__((always_inline)) { keep(j, won); });
  } else {
    auto score32 = [&](int i) __attribute__((always_inline)) {
      const float v = x[i];
      return (a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504088896341f)) : v) + a.bias[l + 16 * i];
    };
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = l + 16 * i < a.E ? key_of(score32(i)) : 0u;
    float before = INFINITY;
    bool close = false;
    take_largest<VPL>(key, l, a.k < a.E ? a.k + 1 : a.k, [&](int j, uint32_t top, int won) __attribute__((always_inline)) {
      const float v = value_of(top);
      const float apart = 16.0f * 0x1p-24f + 4.0f * 0x1p-24f * (fabsf(v) + fabsf(before));
      if (j > 0) close |= !(before - v > apart);      // NaN and infinities too
      before = v;
      if (j < a.k) keep(j, won);
    });
    if (__any(close)) {
      // in 64 bits: those alone that may be among the chosen, so not below the last by more than the error
      const float least = before - 16.0f * 0x1p-24f - 8.0f * 0x1p-24f * fabsf(before);
      uint64_t exact[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        exact[i] = 0;
        if (l + 16 * i < a.E && !(score32(i) < least)) {
          const double v = x[i], score = a.sigmoid ? 1.0 / (1.0 + exp(-v)) : v;
          exact[i] = key_of(score + (double)a.bias[l + 16 * i]);
        }
      }
      take_largest<VPL>(exact, l, a.k, [&](int j, uint64_t, int won) __attribute__((always_inline)) { keep(j, won); });
    }
  }
  const bool there[2] = {l < a.k, 16 + l < a.k};
  float v[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) v[s] = there[s] ? to_f32(row[index[s]]) : -INFINITY;
  if (a.sigmoid) {
    sigmoids(v, there, a.normalise, a.scale, weight);
  } else {
    float p[2], sum;
    // the weights of the chosen alone need their own largest; a row of -inf has no weight
    float top = fmaxf(v[0], v[1]);
    if (!a.normalise) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) top = fmaxf(top, x[i]);
    }
    top = row_max(top);
    const float least = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int s = 0; s < 2; ++s) p[s] = there[s] ? expf(v[s] - least) : 0.0f;
    sum = p[0] + p[1];
    if (!a.normalise) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += expf(x[i] - least);   // exp(-inf) past the last
    }
    sum = row_sum(sum);
#pragma unroll
    for (int s = 0; s < 2; ++s) weight[s] = sum == 0.0f ? 0.0f : p[s] / sum * a.scale;
  }
}

__device__ __forceinline__ int bucket_of(const SortArgs& a, int expert) {
  const uint32_t e = (uint32_t)expert - (uint32_t)a.first;
  return e < (uint32_t)a.count ? (int)e : a.count;
}

constexpr int kSortThreads = 512, kSortWaves = kSortThreads / 64;
constexpr int kBuckets = kMostExperts + 1;
constexpr int kSmallPairs = 1024;          // sorted by one workgroup, by the router's own

// Row of the counts in memory: whole 16 bytes.
__host__ __device__ constexpr int hist_pitch(int buckets) { return (buckets + 3) / 4 * 4; }

struct SortLds {
  int cur[kSortWaves][kBuckets];           // next place of a wave's pairs in a bucket
  int start[kBuckets];
  int sums[kSortWaves];
};

// Exclusive sums of start[0 .. buckets) over the workgroup, in place; -> the last but one's end.
__device__ __forceinline__ void scan_starts(SortLds& s, int buckets) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kPer = (kBuckets + kSortThreads - 1) / kSortThreads;
  int v[kPer], own = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    v[i] = e < buckets ? s.start[e] : 0;
    own += v[i];
  }
  int upto = own;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int x = __shfl_up(upto, m);
    upto += lane >= m ? x : 0;
  }
  if (lane == 63) s.sums[wave] = upto;
  __syncthreads();
  int run = upto - own;
  for (int w = 0; w < wave; ++w) run += s.sums[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < buckets) s.start[e] = run;
    run += v[i];
  }
  __syncthreads();
}

// Counts of the workgroup's pairs [lo, hi) by wave and bucket; bucket(p) tells a pair's.
template <class F>
__device__ __forceinline__ void count_pairs(SortLds& s, int64_t lo, int64_t hi, int64_t step, int buckets,
                                            F bucket) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < kSortWaves * buckets; e += kSortThreads) s.cur[e / buckets][e % buckets] = 0;
  __syncthreads();
  const int64_t from = lo + wave * step, to = from + step < hi ? from + step : hi;
  for (int64_t p = from + lane; p < to; p += 64) atomicAdd(&s.cur[wave][bucket(p)], 1);
  __syncthreads();
}

// Places of the pairs: start[] holds where the workgroup's pairs of a bucket begin, cur[] its
// waves' counts.  A wave takes 64 pairs at a time; those of a bucket find each other by the bits
// of its number.
template <class F>
__device__ __forceinline__ void place_pairs(const SortArgs& a, SortLds& s, int64_t lo, int64_t hi, int64_t step,
                                            int buckets, F bucket) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < buckets; e += kSortThreads) {
    int run = s.start[e];
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = s.cur[w][e];
      s.cur[w][e] = run;
      run += c;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(buckets);
  const int64_t from = lo + wave * step, to = from + step < hi ? from + step : hi;
  volatile int* cur = s.cur[wave];
  for (int64_t p0 = from; p0 < to; p0 += 64) {
    const int64_t p = p0 + lane;
    const bool in = p < to;
    const int b = in ? bucket(p) : 0;
    uint64_t same = __ballot(in);
    for (int i = 0; i < bits; ++i) {
      const uint64_t set = __ballot((b >> i) & 1);
      same &= (b >> i) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    const int at = in ? cur[b] + rank : 0;
    __builtin_amdgcn_wave_barrier();
    if (in && rank == 0) cur[b] = at + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (in) {
      a.order[at] = (int32_t)p;
      a.place[p] = at;
    }
  }
}

// All pairs in one workgroup.
template <class F>
__device__ __forceinline__ void sort_alone(const SortArgs& a, SortLds& s, F bucket) {
  const int buckets = a.count + 1;
  const int64_t step = ((a.n + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  count_pairs(s, 0, a.n, step, buckets, bucket);
  for (int e = threadIdx.x; e < buckets; e += kSortThreads) {
    int all = 0;
    for (int w = 0; w < kSortWaves; ++w) all += s.cur[w][e];
    s.start[e] = all;
  }
  __syncthreads();
  scan_starts(s, buckets);
  for (int e = threadIdx.x; e < buckets; e += kSortThreads) a.offsets[e] = s.start[e];
  place_pairs(a, s, 0, a.n, step, buckets, bucket);
}

__global__ __launch_bounds__(kSortThreads) void sort_alone_kernel(SortArgs a) {
  __shared__ SortLds s;
  sort_alone(a, s, [&](int64_t p) { return bucket_of(a, a.experts[p]); });
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ int hist[kBuckets];
  const int buckets = a.count + 1;
  for (int e = threadIdx.x; e < buckets; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * a.per, hi = lo + a.per < a.n ? lo + a.per : a.n;
  for (int64_t p = lo + threadIdx.x; p < hi; p += kSortThreads) atomicAdd(&hist[bucket_of(a, a.experts[p])], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < buckets; e += kSortThreads) a.hist[blockIdx.x * hist_pitch(buckets) + e] = hist[e];
}

// Every workgroup sums the counts of all of them, and of those before it.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  __shared__ SortLds s;
  __shared__ int before[kBuckets];
  const int buckets = a.count + 1;
  const int64_t lo = blockIdx.x * a.per, hi = lo + a.per < a.n ? lo + a.per : a.n;
  const int64_t step = ((a.per + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  auto bucket = [&](int64_t p) { return bucket_of(a, a.experts[p]); };
  for (int e = threadIdx.x; e < buckets; e += kSortThreads) s.start[e] = before[e] = 0;
  __syncthreads();
  {
    // four buckets a thread, as many threads to each four as there are (what is past the last is not
    // counted)
    const int pitch = hist_pitch(buckets), fours = pitch / 4;
    const int parts = kSortThreads / fours, part = (int)threadIdx.x / fours, e = 4 * ((int)threadIdx.x % fours);
    i32x4 all = {0, 0, 0, 0}, less = {0, 0, 0, 0};
    if (part < parts) {
#pragma unroll 8
      for (int b = part; b < a.blocks; b += parts) {
        const i32x4 c = *(const i32x4*)(a.hist + (int64_t)b * pitch + e);
        all += c;
        less += b < (int)blockIdx.x ? c : i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < buckets) {
          atomicAdd(&s.start[e + i], all[i]);
          atomicAdd(&before[e + i], less[i]);
        }
    }
  }
  count_pairs(s, lo, hi, step, buckets, bucket);
  scan_starts(s, buckets);
  for (int e = threadIdx.x; e < buckets; e += kSortThreads) {
    if (blockIdx.x == 0) a.offsets[e] = s.start[e];
    s.start[e] += before[e];
  }
  __syncthreads();
  place_pairs(a, s, lo, hi, step, buckets, bucket);
}

template <class T, int VPL, bool BIAS>
__device__ __forceinline__ void route_tokens(const RouteArgs& a, int64_t lo, int64_t hi, int* hist, int* buckets) {
  typedef typename T::storage S;
  const int l = threadIdx.x & 15, row = threadIdx.x >> 4, rows = blockDim.x >> 4;
  for (int64_t t0 = lo; t0 < hi; t0 += rows) {
    const int64_t t = t0 + row;
    const bool in = t < hi;
    int index[2];
    float weight[2];
    route_token<S, VPL, BIAS>(a, (const S*)a.logits + (in ? t : lo) * a.stride, l, index, weight);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int j = 16 * s + l;
      if (!in || j >= a.k) continue;
      const int64_t p = t * a.k + j;
      a.experts[p] = index[s];
      a.weights[p] = weight[s];
      if (hist) atomicAdd(&hist[bucket_of(a.s, index[s])], 1);
      if (buckets) buckets[p] = bucket_of(a.s, index[s]);
    }
  }
}

// A workgroup's tokens, and how many pairs of them a bucket has.
template <int VPL>
constexpr int kRouteThreads = VPL <= 16 ? 1024 : 512;     // registers
template <class T, int VPL, bool BIAS>
__global__ __launch_bounds__(kRouteThreads<VPL>) void route_kernel(RouteArgs a, int64_t per) {
  __shared__ int hist[kBuckets];
  const int buckets = a.s.count + 1;
  const bool sorted = a.s.offsets != nullptr;
  if (sorted) {
    for (int e = threadIdx.x; e < buckets; e += kRouteThreads<VPL>) hist[e] = 0;
    __syncthreads();
  }
  const int64_t lo = blockIdx.x * per, hi = lo + per < a.T ? lo + per : a.T;
  route_tokens<T, VPL, BIAS>(a, lo, hi, sorted ? hist : nullptr, nullptr);
  if (!sorted) return;
  __syncthreads();
  for (int e = threadIdx.x; e < buckets; e += kRouteThreads<VPL>) a.s.hist[blockIdx.x * hist_pitch(buckets) + e] = hist[e];
}

// Few tokens: routed and sorted by one workgroup.
template <class T, int VPL, bool BIAS>
__global__ __launch_bounds__(kSortThreads) void route_alone_kernel(RouteArgs a) {
  __shared__ SortLds s;
  __shared__ int pairs[kSmallPairs];
  route_tokens<T, VPL, BIAS>(a, 0, a.T, nullptr, pairs);
  __syncthreads();
  sort_alone(a.s, s, [&](int64_t p) { return pairs[p]; });
}

// A wave's: up to 64 pairs, each of which counts those before it.
template <class T, int VPL, bool BIAS>
__global__ __launch_bounds__(64) void route_tiny_kernel(RouteArgs a) {
  __shared__ int pairs[64];
  const int lane = threadIdx.x, n = (int)a.s.n;
  route_tokens<T, VPL, BIAS>(a, 0, a.T, nullptr, pairs);
  __syncthreads();
  const int b = lane < n ? pairs[lane] : INT32_MAX;
  int at = 0;
  for (int p = 0; p < n; ++p) {
    const int other = __builtin_amdgcn_readlane(b, p);
    at += other < b || (other == b && p < lane);
  }
  if (lane < n) {
    a.s.order[at] = lane;
    a.s.place[lane] = at;
  }
  for (int e = lane; e <= a.s.count; e += 64) {
    int before = 0;
    for (int p = 0; p < n; ++p) before += __builtin_amdgcn_readlane(b, p) < e;
    a.s.offsets[e] = before;
  }
}

// dlogits of one token by 16 lanes.
template <class T>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a) {
  typedef typename T::storage S;
  const int l = threadIdx.x & 15;
  const int64_t t = (((int64_t)a.first_block + blockIdx.x) * 256 + threadIdx.x) >> 4;
  const bool in = t < a.T;
  const S* row = (const S*)a.logits + (in ? t : 0) * a.stride;
  const int64_t p0 = (in ? t : 0) * a.k;
  float top = -INFINITY, all = 0.0f;
  if (!a.sigmoid) {
    if (a.normalise) {
      for (int j = l; j < a.k; j += 16) {
        const int e = a.experts[p0 + j];
        top = fmaxf(top, (uint32_t)e < (uint32_t)a.E ? to_f32(row[e]) : -INFINITY);
      }
    } else {
      for (int c = l; c < a.E; c += 16) top = fmaxf(top, to_f32(row[c]));
    }
    top = row_max(top);
    top = top == -INFINITY ? 0.0f : top;
    if (!a.normalise) {
      for (int c = l; c < a.E; c += 16) all += expf(to_f32(row[c]) - top);
      all = row_sum(all);
    }
  }
  // choice j in lane j % 16: probability, gradient, and how it goes on to the logit
  float p[2], g[2], v[2], dot = 0.0f;
  int index[2];
  bool ok[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int j = 16 * s + l;
    index[s] = j < a.k ? a.experts[p0 + j] : -1;
    ok[s] = (uint32_t)index[s] < (uint32_t)a.E;
    index[s] = ok[s] ? index[s] : -1;
    v[s] = ok[s] ? to_f32(row[index[s]]) : -INFINITY;
    g[s] = ok[s] ? a.dweights[p0 + j] * a.scale : 0.0f;
  }
  if (a.sigmoid) {
    sigmoids(v, ok, a.normalise, 1.0f, p);
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s) p[s] = ok[s] ? expf(v[s] - top) : 0.0f;
    const float sum = a.normalise ? row_sum(p[0] + p[1]) : all;
#pragma unroll
    for (int s = 0; s < 2; ++s) p[s] = sum == 0.0f ? 0.0f : p[s] / sum;
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) dot += ok[s] ? g[s] * p[s] : 0.0f;
  dot = row_sum(dot);
  float d[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    // normalised, both: q (g - sum g q), times 1 - p where q are shares of sigmoids; softmax over
    // all: p g here and - p sum g p for every expert below
    d[s] = p[s] * (a.normalise ? g[s] - dot : g[s]);
    if (a.sigmoid) d[s] *= index[s] >= 0 ? 1.0f / (1.0f + expf(to_f32(row[index[s]]))) : 0.0f;
  }
  const bool spread = !a.sigmoid && !a.normalise;
  S* out = (S*)a.dlogits + t * a.E;
  for (int c0 = 0; c0 < a.E; c0 += 16) {
    const int c = c0 + l;
    float v = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      const int at = __shfl(j < 16 ? index[0] : index[1], j & 15, 16);
      const float dj = __shfl(j < 16 ? d[0] : d[1], j & 15, 16);
      v += at == c ? dj : 0.0f;
    }
    if (!in || c >= a.E) continue;
    if (spread) v -= all == 0.0f ? 0.0f : expf(to_f32(row[c]) - top) / all * dot;
    out[c] = from_f32<S>(v);
  }
}

// ---- rows there and back ------------------------------------------------------------------
constexpr int kRun = 8;                    // columns that a thread takes at a time
constexpr int kTogether = 8;               // choices whose rows are in flight together

// WHOLE: C is a multiple of a run, and no load stands under a condition (the same combine_kernel as
// below 52 us, 57 with the test at each run).
template <bool WHOLE, class S>
__device__ __forceinline__ Run<kRun, S> load_part(const S* p, int left) {
  if (WHOLE || left >= kRun) return load_run<kRun>(p);
  Run<kRun, S> r;
#pragma unroll
  for (int i = 0; i < kRun; ++i) r.v[i] = i < left ? p[i] : (S)0.0f;
  return r;
}
template <bool WHOLE, class S>
__device__ __forceinline__ void store_part(S* p, const float* x, int left) {
  if (WHOLE || left >= kRun) return store_run<kRun>(p, x);
#pragma unroll
  for (int i = 0; i < kRun; ++i)
    if (i < left) p[i] = from_f32<S>(x[i]);
}

// The token and the run of columns of a thread: several tokens to a workgroup where rows are short,
// several workgroups to a token where they are long, so that no thread waits for memory twice (4095
// tokens of 6 rows of 4096 columns in fp16: combine_kernel 57 us, 65 with two runs a thread).
struct Part {
  int64_t t, c;         // token, first column
  int left;             // columns from there on, at most kRun
  bool in;
  __device__ __forceinline__ Part(const RowsArgs& a) {
    const uint32_t runs = (uint32_t)((a.C + kRun - 1) / kRun), blocks = (runs + 255) / 256;
    const uint64_t block = (uint64_t)a.first_block + blockIdx.x;
    uint32_t v;
    if (runs < 256) {
      const uint32_t tokens = 256 / runs, r = threadIdx.x / runs;
      t = (int64_t)block * tokens + r;
      v = threadIdx.x % runs;
      in = r < tokens && t < a.T;
    } else {
      t = (int64_t)(block / blocks);
      v = (uint32_t)(block % blocks) * 256 + threadIdx.x;
      in = v < runs;
    }
    c = (int64_t)v * kRun;
    left = (int)(a.C - c < kRun ? a.C - c : kRun);
  }
};
int64_t part_blocks(int64_t T, int64_t C) {
  const int64_t runs = (C + kRun - 1) / kRun;
  return runs < 256 ? (T + 256 / runs - 1) / (256 / runs) : T * ((runs + 255) / 256);
}

// rows[place] = weight tokens[t], 0 where the expert is elsewhere. A token is read once for all of
// its choices. Bound by memory, its writes above all: 8191 tokens of 2048 columns in bf16 to 8
// places, 302 MB, 49 us, 6.1 TB/s (a call 51 where the same tensors come again, 58 with others).
template <class T, bool WHOLE>
__global__ __launch_bounds__(256) void gather_kernel(RowsArgs a) {
  typedef typename T::storage S;
  const Part u(a);
  if (!u.in) return;
  const int64_t n = a.T * a.k;
  const int kept = a.offsets[a.count];
  const Run<kRun, S> r = load_part<WHOLE>((const S*)a.tokens + u.t * a.stride + u.c, u.left);
  float x[kRun], y[kRun];
  widen(r, x);
  for (int j = 0; j < a.k; ++j) {
    const int64_t p = u.t * a.k + j;
    const int at = a.place[p];
    if ((uint64_t)(int64_t)at >= (uint64_t)n) continue;
    const bool here = at < kept;
    const float w = a.weights ? a.weights[p] : 1.0f;
#pragma unroll
    for (int i = 0; i < kRun; ++i) y[i] = here ? x[i] * w : 0.0f;
    store_part<WHOLE>((S*)a.out + at * a.C + u.c, y, u.left);
  }
}

// out[t] = tokens[t] + sum_j weight rows[place], in the order of the choices. Bound by memory: 4095
// tokens of 6 rows of 4096 columns in fp16, 235 MB, 52 us, 4.5 TB/s.
template <class T, class TO, bool WHOLE>
__global__ __launch_bounds__(256, 4) void combine_kernel(RowsArgs a) {
  typedef typename T::storage S;
  typedef typename TO::storage SO;
  const Part u(a);
  if (!u.in) return;
  const int kept = a.offsets[a.count];
  const int64_t n = a.T * a.k, most = kept < n ? kept : n;
  float y[kRun] = {};
  if (a.tokens) widen(load_part<WHOLE>((const SO*)a.tokens + u.t * a.stride + u.c, u.left), y);
  for (int j0 = 0; j0 < a.k; j0 += kTogether) {
    Run<kRun, S> r[kTogether];
    float w[kTogether];
    int at[kTogether];
    bool here[kTogether];
    // places first, then rows: memory answers in order
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const int64_t p = u.t * a.k + (j0 + j < a.k ? j0 + j : 0);
      at[j] = a.place[p];
      w[j] = a.weights ? a.weights[p] : 1.0f;
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      here[j] = j0 + j < a.k && at[j] >= 0 && at[j] < most;
      // a row that nobody has is not read: the first stands in for it and does not count
      if (j0 + j < a.k) r[j] = load_part<WHOLE>((const S*)a.rows + (here[j] ? at[j] : 0) * a.C + u.c, u.left);
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      if (!here[j]) continue;
      float x[kRun];
      widen(r[j], x);
#pragma unroll
      for (int i = 0; i < kRun; ++i) y[i] = fmaf(w[j], x[i], y[i]);
    }
  }
  store_part<WHOLE>((SO*)a.out + u.t * a.C + u.c, y, u.left);
}

// Sorted rows of tokens as gather_kernel, and the product of every pair's token and row; a
// workgroup a token, since a product is over all of its columns. Bound by memory: the size of
// combine_kernel, 436 MB, 89 us, 4.9 TB/s.
template <class TT, class T, bool WHOLE>
__global__ __launch_bounds__(256) void combine_grad_kernel(RowsArgs a) {
  typedef typename TT::storage ST;
  typedef typename T::storage S;
  __shared__ float sums[4][kTogether];
  const int64_t t = (int64_t)a.first_block + blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n = a.T * a.k;
  const int kept = a.offsets[a.count];
  const int runs = (int)((a.C + kRun - 1) / kRun);
  for (int j0 = 0; j0 < a.k; j0 += kTogether) {
    float dot[kTogether] = {};
    int at[kTogether];
    float w[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const bool in = j0 + j < a.k;
      const int64_t p = t * a.k + (in ? j0 + j : 0);
      at[j] = in ? a.place[p] : -1;
      at[j] = (uint64_t)(int64_t)at[j] < (uint64_t)n ? at[j] : -1;
      w[j] = a.weights ? a.weights[p] : 1.0f;
    }
    for (int v = tid; v < runs; v += 256) {
      const int64_t c = (int64_t)v * kRun;
      const int left = (int)(a.C - c < kRun ? a.C - c : kRun);
      Run<kRun, S> r[kTogether];
      if (a.dots) {
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
          if (at[j] >= 0 && at[j] < kept) r[j] = load_part<WHOLE>((const S*)a.rows + at[j] * a.C + c, left);
      }
      float d[kRun], x[kRun];
      widen(load_part<WHOLE>((const ST*)a.tokens + t * a.stride + c, left), d);
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        if (at[j] < 0) continue;
        const bool here = at[j] < kept;
        if (a.dots && here) {
          widen(r[j], x);
#pragma unroll
          for (int i = 0; i < kRun; ++i) dot[j] = fmaf(d[i], x[i], dot[j]);
        }
        if (a.out) {
#pragma unroll
          for (int i = 0; i < kRun; ++i) x[i] = here ? d[i] * w[j] : 0.0f;
          store_part<WHOLE>((S*)a.out + at[j] * a.C + c, x, left);
        }
      }
    }
    if (!a.dots) continue;
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) dot[j] += __shfl_xor(dot[j], m);
      if (lane == 0) sums[wave][j] = dot[j];
    }
    __syncthreads();
    if (tid < kTogether && j0 + tid < a.k)
      a.dots[t * a.k + j0 + tid] = (sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid]);
    __syncthreads();
  }
}

template <class F>
hipError_t by_type(awq_dtype_t dt, F f) {
  if (dt == AWQ_F32) f(F32T{});
  else if (dt == AWQ_F16) f(F16T{});
  else f(BF16T{});
  return hipGetLastError();
}

template <class F>
void by_whole(int64_t C, F f) {
  if (C % kRun == 0) f(std::true_type{});
  else f(std::false_type{});
}

// Workgroups that share the pairs; each sums all their counts, so not more than the chip takes at once.
int sort_blocks(int64_t n) { return (int)std::min<int64_t>(256, (n + 511) / 512); }

template <class T, int VPL, bool BIAS>
void go_bias(const RouteArgs& a, bool alone, int64_t per, int blocks, hipStream_t st) {
  if (!alone) route_kernel<T, VPL, BIAS><<<blocks, kRouteThreads<VPL>, 0, st>>>(a, per);
  else if (a.s.n <= 64) route_tiny_kernel<T, VPL, BIAS><<<1, 64, 0, st>>>(a);
  else route_alone_kernel<T, VPL, BIAS><<<1, kSortThreads, 0, st>>>(a);
}

template <class T, int VPL>
void go_route(const RouteArgs& a, bool alone, int64_t per, int blocks, hipStream_t st) {
  if (a.bias) go_bias<T, VPL, true>(a, alone, per, blocks, st);
  else go_bias<T, VPL, false>(a, alone, per, blocks, st);
}

}  // namespace

size_t moe_sort_ws_bytes(int64_t n, int count) {
  return n <= kSmallPairs ? 0 : (size_t)sort_blocks(n) * hist_pitch(count + 1) * 4;
}

hipError_t launch_moe_sort(SortArgs a, hipStream_t st) {
  ProfScope prof("awq_moe_sort", st);
  if (a.n <= kSmallPairs) {
    sort_alone_kernel<<<1, kSortThreads, 0, st>>>(a);
    return hipGetLastError();
  }
  a.blocks = sort_blocks(a.n);
  a.per = (a.n + a.blocks - 1) / a.blocks;
  sort_count_kernel<<<a.blocks, kSortThreads, 0, st>>>(a);
  sort_place_kernel<<<a.blocks, kSortThreads, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_moe_route(RouteArgs a, awq_dtype_t dt, hipStream_t st) {
  ProfScope prof("awq_moe_route", st);
  const bool sorted = a.s.offsets != nullptr;
  a.s.n = a.T * a.k;
  a.s.experts = a.experts;
  const bool alone = sorted && a.s.n <= kSmallPairs;
  // a workgroup's pairs are whole tokens
  int64_t blocks = sorted ? sort_blocks(a.s.n) : (a.T + 31) / 32;
  blocks = std::min<int64_t>(std::max<int64_t>(blocks, 1), 1 << 20);
  const int64_t per = std::max<int64_t>(1, (a.T + blocks - 1) / blocks);
  blocks = (a.T + per - 1) / per;
  a.s.blocks = (int)blocks;
  a.s.per = per * a.k;
  const hipError_t e = by_type(dt, [&](auto t) {
    typedef decltype(t) T;
    if (a.E <= 64) go_route<T, 4>(a, alone, per, (int)blocks, st);
    else if (a.E <= 128) go_route<T, 8>(a, alone, per, (int)blocks, st);
    else if (a.E <= 256) go_route<T, 16>(a, alone, per, (int)blocks, st);
    else if (a.E <= 512) go_route<T, 32>(a, alone, per, (int)blocks, st);
    else go_route<T, 64>(a, alone, per, (int)blocks, st);
  });
  if (e != hipSuccess || !sorted || alone) return e;
  sort_place_kernel<<<a.s.blocks, kSortThreads, 0, st>>>(a.s);
  return hipGetLastError();
}

hipError_t launch_moe_route_grad(RouteGradArgs a, awq_dtype_t dt, hipStream_t st) {
  ProfScope prof("awq_moe_route_grad", st);
  return by_type(dt, [&](auto t) {
    in_parts((a.T + 15) / 16, 256, [&](uint32_t first, unsigned grid) {
      a.first_block = first;
      route_grad_kernel<decltype(t)><<<grid, 256, 0, st>>>(a);
    });
  });
}

hipError_t launch_moe_gather(RowsArgs a, awq_dtype_t dt, hipStream_t st) {
  ProfScope prof("awq_moe_gather", st);
  return by_type(dt, [&](auto t) {
    by_whole(a.C, [&](auto whole) {
      in_parts(part_blocks(a.T, a.C), 256, [&](uint32_t first, unsigned grid) {
        a.first_block = first;
        gather_kernel<decltype(t), decltype(whole)::value><<<grid, 256, 0, st>>>(a);
      });
    });
  });
}

hipError_t launch_moe_combine(RowsArgs a, awq_dtype_t dt, awq_dtype_t out_dt, hipStream_t st) {
  ProfScope prof("awq_moe_combine", st);
  hipError_t e = hipSuccess;
  const hipError_t f = by_type(dt, [&](auto t) {
    e = by_type(out_dt, [&](auto o) {
      by_whole(a.C, [&](auto whole) {
        in_parts(part_blocks(a.T, a.C), 256, [&](uint32_t first, unsigned grid) {
          a.first_block = first;
          combine_kernel<decltype(t), decltype(o), decltype(whole)::value><<<grid, 256, 0, st>>>(a);
        });
      });
    });
  });
  return e != hipSuccess ? e : f;
}

hipError_t launch_moe_combine_grad(RowsArgs a, awq_dtype_t token_dt, awq_dtype_t dt, hipStream_t st) {
  ProfScope prof("awq_moe_combine_grad", st);
  hipError_t e = hipSuccess;
  const hipError_t f = by_type(token_dt, [&](auto t) {
    e = by_type(dt, [&](auto r) {
      by_whole(a.C, [&](auto whole) {
        in_parts(a.T, 256, [&](uint32_t first, unsigned grid) {
          a.first_block = first;
          combine_grad_kernel<decltype(t), decltype(r), decltype(whole)::value><<<grid, 256, 0, st>>>(a);
        });
      });
    });
  });
  return e != hipSuccess ? e : f;
}

}  // namespace awq
