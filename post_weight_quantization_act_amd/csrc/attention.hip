// Attention over the paged 8-bit cache.
//
//   o = sum_j p_j v_j,  p = softmax_j(scale q . k_j)  over the tokens j that the row sees,
//   k_j = (u - 128) step of its page and head, v_j likewise.
// A row that sees nothing gives 0, and -inf for the logarithm of its sum.
#include "kv.h"

namespace awq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_reduce(float v, bool sum, float* red) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const float o = __shfl_xor(v, m);
    v = sum ? v + o : fmaxf(v, o);
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kThreads / 64; ++w) v = sum ? v + red[w] : fmaxf(v, red[w]);
  return v;
}

// One workgroup for each row and query head, one token a lane.
template <class T>
__global__ __launch_bounds__(kThreads) void attention_kernel(AttArgs a) {
  typedef typename T::storage S;
  __shared__ float qs[256], ps[kThreads], red[kThreads / 64];
  const KvArgs& c = a.c;
  int64_t g = blockIdx.x;
  const int hq = (int)(g % a.Hq);
  g /= a.Hq;
  const int i = (int)(g % a.max_new), b = (int)(g / a.max_new);
  int64_t row0;
  int n;
  rows_of(c, b, row0, n);
  if (i >= n) return;
  const int tid = threadIdx.x, h = hq / (a.Hq / c.Hkv), len = a.lens[b];
  int lo, hi;
  seen_by(a, len, n, i, lo, hi);
  const S* q = (const S*)a.q + (row0 + i) * a.qs[0] + hq * a.qs[1];
  if (tid < c.D) qs[tid] = to_f32(q[tid]);
  __syncthreads();
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int t0 = lo; t0 < hi; t0 += kThreads) {
    const int t = t0 + tid;
    const int id = t < hi ? page_id(c, b, t >> c.p_shift) : -1;
    float s = -INFINITY;
    float vstep = 0.0f;
    if (id >= 0) {
      const int64_t blk = (int64_t)id * c.Hkv + h;
      const uint8_t* k = c.k_codes + (blk * c.P + (t & (c.P - 1))) * c.D;
      float dot = 0.0f;
      for (int d = 0; d < c.D; ++d) dot += qs[d] * (float)((int)k[d] - 128);
      s = dot * c.k_steps[blk] * a.scale;
      vstep = c.v_steps[blk];
    }
    const float top = fmaxf(m, block_reduce(s, false, red));
    const float ref = top == -INFINITY ? 0.0f : top;
    const float p = id >= 0 ? __expf(s - ref) : 0.0f;
    const float keep = __expf(m - ref);
    l = l * keep + block_reduce(p, true, red);
    o *= keep;
    m = top;
    ps[tid] = id >= 0 ? p * vstep : 0.0f;
    __syncthreads();
    if (tid < c.D) {
      const int count = hi - t0 < kThreads ? hi - t0 : kThreads;
      for (int j = 0; j < count; ++j) {
        const int id2 = page_id(c, b, (t0 + j) >> c.p_shift);
        if (id2 < 0) continue;
        const uint8_t* v = c.v_codes + (((int64_t)id2 * c.Hkv + h) * c.D + tid) * c.P;
        o += ps[j] * (float)((int)v[(t0 + j) & (c.P - 1)] - 128);
      }
    }
    __syncthreads();
  }
  const int64_t r = (row0 + i) * a.Hq + hq;
  if (tid < c.D) ((S*)a.out)[r * c.D + tid] = from_f32<S>(l == 0.0f ? 0.0f : o / l);
  if (tid == 0 && a.lse) a.lse[r] = l == 0.0f ? -INFINITY : m + __logf(l);
}

}  // namespace

size_t kv_attention_ws_bytes(int64_t, int64_t, int, int, int, int, int) { return 0; }

int64_t kv_attention_blocks(int64_t, int64_t B, int Hq, int, int, int max_new, int) {
  return max_new > INT64_MAX / Hq / B ? INT64_MAX : B * max_new * Hq;
}

hipError_t launch_kv_attention(const AttArgs& a, awq_dtype_t dt, void*, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)a.c.B * a.max_new * a.Hq);
  ProfScope prof("awq_kv_attention", st);
  if (dt == AWQ_F16) attention_kernel<F16T><<<grid, kThreads, 0, st>>>(a);
  else attention_kernel<BF16T><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace awq
