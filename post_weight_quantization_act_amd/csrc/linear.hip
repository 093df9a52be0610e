// y = act(x W'^T + bias) [times (x W_up'^T + bias_up)] + residual with packed W' = (c - z) step:
// one projection for all rows, or each expert's own for its sorted rows.
//
// The codes' layout is awq_lowbit_repack's: the words of row n's chunk j (32 columns) at
// (j R + n) bits, R the rows of all experts; (step, z) of group g at g R + n.  Codes become the
// exact integers c - z in the activations' type, in the registers that the matrix
// instructions read them from; products are exact and sums are held in fp32, by group, scaled by
// the group's step.
#ifndef AWQ_LINEAR_BITS
#error "compiled once for each width of codes"
#endif

#include "linear.h"

namespace awq {
namespace {

constexpr int BITS = AWQ_LINEAR_BITS;

// ---- rows of a tile --------------------------------------------------------------------
struct Tile {
  int64_t row0;      // first output row
  int rows;          // 0: there is no such tile
  int expert;        // `experts`: rows that no expert here has
};

// Tile `want` of the rows, `most` rows each, expert by expert; the wave's 64 lanes look at
// 64 experts at a time.
__device__ __forceinline__ Tile find_tile(const LinearArgs& a, int most, int64_t want) {
  Tile t;
  if (!a.offsets) {
    t.row0 = want * most;
    const int64_t left = a.rows - t.row0;
    t.rows = left < 0 ? 0 : (int)(left < most ? left : most);
    t.expert = 0;
    return t;
  }
  const int lane = threadIdx.x & 63, total = (int)a.rows;
  int before = 0;
  for (int e0 = 0; e0 <= a.experts; e0 += 64) {
    const int e = e0 + lane;
    int lo = e <= a.experts ? a.offsets[e] : total;
    int hi = e < a.experts ? a.offsets[e + 1] : total;
    lo = lo < 0 ? 0 : lo > total ? total : lo;
    hi = hi < lo ? lo : hi > total ? total : hi;
    const int tiles = (hi - lo + most - 1) / most;
    int upto = tiles;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int x = __shfl_up(upto, m);
      upto += lane >= m ? x : 0;
    }
    const uint64_t mine = __ballot(want < before + upto);
    if (mine) {
      const int l = __builtin_ctzll(mine);
      const int part = (int)want - (before + __builtin_amdgcn_readlane(upto - tiles, l));
      const int from = __builtin_amdgcn_readlane(lo, l), to = __builtin_amdgcn_readlane(hi, l);
      t.row0 = from + (int64_t)part * most;
      t.rows = to - (int)t.row0 < most ? to - (int)t.row0 : most;
      t.expert = e0 + l;
      return t;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return Tile{0, 0, 0};
}

// Row of x that output row r takes.
__device__ __forceinline__ int64_t source(const LinearArgs& a, int64_t r) {
  if (!a.order) return r;
  const int64_t s = (uint32_t)a.order[r] / (uint32_t)a.per_token;
  return s < a.x_rows ? s : 0;
}

// ---- epilogue ------------------------------------------------------------------------------
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case AWQ_ACT_RELU: return v < 0.0f ? 0.0f : v;
    case AWQ_ACT_SILU: return v / (1.0f + expf(-v));
    case AWQ_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case AWQ_ACT_GELU_TANH: return 0.5f * v * (1.0f + tanhf(0.79788456080286536f * (v + 0.044715f * v * v * v)));
    default: return v;
  }
}

__device__ __forceinline__ float load_as(const void* p, int64_t i, int type) {
  if (type == AWQ_F32) return ((const float*)p)[i];
  return type == AWQ_F16 ? (float)((const _Float16*)p)[i] : (float)((const __bf16*)p)[i];
}
__device__ __forceinline__ void store_as(void* p, int64_t i, int type, float v) {
  if (type == AWQ_F32) ((float*)p)[i] = v;
  else if (type == AWQ_F16) ((_Float16*)p)[i] = (_Float16)v;
  else ((__bf16*)p)[i] = (__bf16)v;
}

// Output (row, column n) of an expert from its sums, gate and up where gated.
__device__ __forceinline__ void finish(const LinearArgs& a, int expert, int64_t row, int n, float v, float up) {
  const int outputs = a.gated ? a.N / 2 : a.N;
  if (a.bias) {
    const float* b = a.bias + (int64_t)expert * a.N;
    v += b[n];
    if (a.gated) up += b[outputs + n];
  }
  v = activate(v, a.act);
  if (a.gated) v *= up;
  if (a.residual) v += load_as(a.residual, row * a.residual_stride + n, a.out_type);
  store_as(a.out, row * outputs + n, a.out_type, v);
}

// ---- codes to values ------------------------------------------------------------------------
// Eight consecutive ones, the Q-th of a run's words, as a fragment.
template <class S, int NW, int Q>
__device__ __forceinline__ i32x4 eight(const uint32_t (&w)[NW], half2v negz, const float* sub,
                                       const QuarterOps<BITS>& ops) {
  return i32x4{small_pair<S, BITS, NW, 4 * Q>(w, negz, sub, ops), small_pair<S, BITS, NW, 4 * Q + 1>(w, negz, sub, ops),
               small_pair<S, BITS, NW, 4 * Q + 2>(w, negz, sub, ops), small_pair<S, BITS, NW, 4 * Q + 3>(w, negz, sub, ops)};
}

struct Zero {
  half2v neg;
  float sub[QuarterWindows<BITS>::kPer];
  __device__ __forceinline__ Zero(float z) {
    const _Float16 n = (_Float16)(-(1024.0f + z));
    neg = half2v{n, n};
#pragma unroll
    for (int t = 0; t < QuarterWindows<BITS>::kPer; ++t) sub[t] = (float)(1 << (23 - BITS * t)) + z;
  }
};

// ---- few rows ---------------------------------------------------------------------------------
// A workgroup takes WT tiles of 16 weight rows (gated: a tile of gates and the same of ups) and
// 16 TT output rows; its waves share the columns of K, 128 at a time, and add up in LDS.  Lane
// 16 g + r holds weight row r and the 32 codes of chunk g of the four: one load of `bits` words;
// instruction i of four multiplies the chunks' codes 8 i .. 8 i + 7.
template <class S, int TT, int WT>
__global__ __launch_bounds__(512, 2) void linear_few_kernel(LinearArgs a, int col_tiles) {
  extern __shared__ __attribute__((aligned(16))) f32x4 red[];      // [waves][WT][TT][64]
  const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int outputs = a.gated ? a.N / 2 : a.N;
  const int wide = a.gated ? 16 : 16 * WT;             // outputs of a workgroup
  const int n0 = (int)(blockIdx.x % (uint32_t)col_tiles) * wide;
  const Tile t = find_tile(a, 16 * TT, blockIdx.x / (uint32_t)col_tiles);
  if (t.rows == 0) return;
  if (t.expert == a.experts) {
    for (int e = tid; e < t.rows * wide; e += blockDim.x)
      if (n0 + e % wide < outputs) store_as(a.out, (t.row0 + e / wide) * outputs + n0 + e % wide, a.out_type, 0.0f);
    return;
  }
  const int chunks = (int)(a.K / 32), steps = (chunks + 3) / 4;
  int64_t wrow[WT];
#pragma unroll
  for (int w = 0; w < WT; ++w) {
    int n = n0 + (a.gated ? 0 : 16 * w) + r;
    n = n < outputs ? n : outputs - 1;
    wrow[w] = (int64_t)t.expert * a.N + n + (a.gated && w ? outputs : 0);
  }
  const S* x[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int m = 16 * i + r;
    x[i] = m < t.rows ? (const S*)a.x + source(a, t.row0 + m) * a.stride : nullptr;
  }
  struct Step {
    uint32_t w[WT][BITS];
    float2 m[WT];
    i32x4 x[TT][4];
  };
  auto load = [&](int s, Step& b) __attribute__((always_inline)) {
    const int j = 4 * s + g;
    const bool in = j < chunks;
    const int64_t jj = in ? j : chunks - 1;
#pragma unroll
    for (int w = 0; w < WT; ++w) {
      const uint32_t* p = a.codes + (jj * a.R + wrow[w]) * BITS;
#pragma unroll
      for (int i = 0; i < BITS; ++i) b.w[w][i] = p[i];
      b.m[w] = a.meta[(jj >> a.lg_cpg) * a.R + wrow[w]];
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        b.x[i][q] = i32x4{0, 0, 0, 0};
        if (x[i] && in) b.x[i][q] = *(const i32x4*)(x[i] + 32 * jj + 8 * q);
      }
  };
  const int apart = a.lg_cpg == 0 ? 4 : a.lg_cpg == 1 ? 2 : 1;   // groups of a step's 128 columns
  const QuarterOps<BITS> ops = magic_ops<BITS, QuarterWindows<BITS>::kPer>();
  f32x4 tot[WT][TT];
#pragma unroll
  for (int w = 0; w < WT; ++w)
#pragma unroll
    for (int i = 0; i < TT; ++i) tot[w][i] = f32x4{0, 0, 0, 0};
  auto multiply = [&](const Step& b) __attribute__((always_inline)) {
#pragma unroll
    for (int w = 0; w < WT; ++w) {
      const Zero z(b.m[w].y);
      const i32x4 f[4] = {eight<S, BITS, 0>(b.w[w], z.neg, z.sub, ops), eight<S, BITS, 1>(b.w[w], z.neg, z.sub, ops),
                          eight<S, BITS, 2>(b.w[w], z.neg, z.sub, ops), eight<S, BITS, 3>(b.w[w], z.neg, z.sub, ops)};
      if (apart == 1) {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          f32x4 acc = {0, 0, 0, 0};
#pragma unroll
          for (int q = 0; q < 4; ++q) acc = mfma16x32<S>(b.x[i][q], f[q], acc);
          tot[w][i] += acc * b.m[w].x;
        }
      } else {
        // several groups in the step: one at a time, the other chunks' activations taken as 0
        for (int part = 0; part < apart; ++part) {
          const int g0 = part * (4 / apart);
          const bool on = g >= g0 && g < g0 + 4 / apart;
          const float d = __shfl(b.m[w].x, 16 * g0 + r);
#pragma unroll
          for (int i = 0; i < TT; ++i) {
            f32x4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) acc = mfma16x32<S>(on ? b.x[i][q] : i32x4{0, 0, 0, 0}, f[q], acc);
            tot[w][i] += acc * d;
          }
        }
      }
    }
  };
  Step cur, next;
  int s = wave;
  if (s < steps) load(s, cur);
  for (; s < steps; s += waves) {
    if (s + waves < steps) load(s + waves, next);
    multiply(cur);
    cur = next;
  }
#pragma unroll
  for (int w = 0; w < WT; ++w)
#pragma unroll
    for (int i = 0; i < TT; ++i) red[((wave * WT + w) * TT + i) * 64 + lane] = tot[w][i];
  __syncthreads();
  // lane l of a tile holds weight row l % 16 and output rows 4 (l / 16) .. + 3
  const float* sums = (const float*)red;
  auto total = [&](int w, int m, int n) {
    float v = 0.0f;
    for (int k = 0; k < waves; ++k)
      v += sums[(((k * WT + w) * TT + (m >> 4)) * 64 + n + 16 * ((m & 15) >> 2)) * 4 + (m & 3)];
    return v;
  };
  for (int e = tid; e < t.rows * wide; e += blockDim.x) {
    const int n = e % wide, m = e / wide;
    if (n0 + n >= outputs) continue;
    const float v = total(a.gated ? 0 : n >> 4, m, n & 15);
    const float up = a.gated ? total(WT - 1, m, n) : 0.0f;
    finish(a, t.expert, t.row0 + m, n0 + n, v, up);
  }
}

// ---- many rows -----------------------------------------------------------------------------------
// A workgroup of four waves takes 32 MT output rows and 256 weight rows, a wave all the output
// rows and 64 weight rows (gated: 32 gates and the same ups).  Activations go through LDS, 128
// columns at a time, two buffers; a wave unpacks its own weights in registers, so each code
// is unpacked once for 32 MT rows: lane half h takes codes 16 h .. 16 h + 15 of a chunk.
// The sums are in units of the group's step U: where the next group begins they are multiplied by
// U / U', a step of 0 leaves the unit as it is and its codes count as 0.
constexpr int kTileWaves = 4;

template <class S, int MT>
__global__ __launch_bounds__(256, 2) void linear_tile_kernel(LinearArgs a, int col_tiles) {
  constexpr int NW = (BITS + 1) / 2;
  constexpr int kRows = 32 * MT, kPer = 2 * MT;                  // transfers of a wave and step
  __shared__ __attribute__((aligned(1024))) char xs[2][kRows * 256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int outputs = a.gated ? a.N / 2 : a.N;
  const int wide = a.gated ? 32 : 64;                            // outputs of a wave
  const int first = (int)(blockIdx.x % (uint32_t)col_tiles) * kTileWaves * wide, n0 = first + wave * wide;
  const Tile t = find_tile(a, kRows, blockIdx.x / (uint32_t)col_tiles);
  if (t.rows == 0) return;
  if (t.expert == a.experts) {
    const int span = kTileWaves * wide;
    for (int e = tid; e < t.rows * span; e += 256)
      if (first + e % span < outputs) store_as(a.out, (t.row0 + e / span) * outputs + first + e % span, a.out_type, 0.0f);
    return;
  }
  const int chunks = (int)(a.K / 32), steps = (chunks + 3) / 4, cmask = (1 << a.lg_cpg) - 1;
  int64_t wrow[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    int n = n0 + (a.gated ? 0 : 32 * w) + r;
    n = n < outputs ? n : outputs - 1;
    wrow[w] = (int64_t)t.expert * a.N + n + (a.gated && w ? outputs : 0);
  }
  // activations: transfer q of a step brings rows 4 q .. 4 q + 3, 16-byte part p of row m from
  // part p ^ (m % 16); rows past the last are the first again
  const i32x4 rx = byte_range(a.x, (uint32_t)(((a.x_rows - 1) * a.stride + a.K) * 2));
  const uint32_t base = (uint32_t)(uintptr_t)&xs[0][0];
  uint32_t xoff[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int m = 4 * (wave * kPer + i) + (lane >> 4);
    const int64_t row = source(a, t.row0 + (m < t.rows ? m : 0));
    xoff[i] = (uint32_t)((row * a.stride + 8 * ((lane & 15) ^ (m & 15))) * 2);
  }
  auto fetch_x = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      to_lds16(rx, base + buf * (kRows * 256) + (wave * kPer + i) * 1024, xoff[i]);
      xoff[i] += 256;
    }
  };
  const int qw = (16 * h * BITS) >> 5, qoff = (16 * h * BITS) & 31;
  struct Codes {
    uint32_t w[2][4][NW];
    float2 m[2][4];
  };
  auto fetch_codes = [&](int s, Codes& c) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t j = 4 * s + q < chunks ? 4 * s + q : chunks - 1;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t* p = a.codes + (j * a.R + wrow[w]) * BITS + qw;
#pragma unroll
        for (int i = 0; i < NW; ++i) c.w[w][q][i] = p[i];
        c.m[w][q] = a.meta[(j >> a.lg_cpg) * a.R + wrow[w]];
      }
    }
  };
  const QuarterOps<BITS> ops = magic_ops<BITS, QuarterWindows<BITS>::kPer>();
  f32x16 acc[MT][2];
  float unit[2] = {1.0f, 1.0f};
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int w = 0; w < 2; ++w) acc[i][w] = f32x16{};
  auto multiply = [&](int s, const Codes& c, const char* xb) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = 4 * s + q;
      if (j >= chunks) break;
      if ((j & cmask) == 0) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float u = c.m[w][q].x != 0.0f ? c.m[w][q].x : unit[w];
          if (j > 0) {
            const float by = unit[w] / u;
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i][w] *= by;
          }
          unit[w] = u;
        }
      }
      i32x4 f[2][2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const bool live = c.m[w][q].x != 0.0f;
        uint32_t run[NW];
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          uint32_t v = c.w[w][q][i];
          if constexpr (BITS % 2 == 1) v = i + 1 < NW ? __builtin_amdgcn_alignbit(c.w[w][q][i + 1 < NW ? i + 1 : i], v, qoff) : v >> qoff;
          run[i] = live ? v : 0u;
        }
        const Zero z(live ? c.m[w][q].y : 0.0f);
        f[w][0] = eight<S, NW, 0>(run, z.neg, z.sub, ops);
        f[w][1] = eight<S, NW, 1>(run, z.neg, z.sub, ops);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int m = 32 * i + r, p = 4 * q + 2 * h + k;
          const i32x4 fa = *(const i32x4*)(xb + m * 256 + 16 * (p ^ (m & 15)));
#pragma unroll
          for (int w = 0; w < 2; ++w) acc[i][w] = mfma32<S>(fa, f[w][k], acc[i][w]);
        }
    }
  };
  Codes cur, next;
  fetch_x(0);
  fetch_codes(0, cur);
  vm_wait<0>();
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    if (s + 1 < steps) {
      fetch_x((s + 1) & 1);
      fetch_codes(s + 1, next);
    }
    multiply(s, cur, xs[s & 1]);
    vm_wait<0>();
    __syncthreads();
    cur = next;
  }
  // Lane l holds weight row l % 32 and output rows 8 (e / 4) + 4 (l / 32) + e % 4.  Sixteen rows at
  // a time go through LDS, so that a wave stores whole rows of its outputs.
  float* turn = (float*)&xs[0][0] + wave * 16 * 64;
  const int span = a.gated ? 32 : 64, col = lane % span;
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int m = 8 * (e >> 2) + 4 * h + (e & 3);
#pragma unroll
      for (int w = 0; w < 2; ++w)
        turn[m * 64 + ((32 * w + r) ^ (32 * h))] = acc[i >> 1][w][8 * (i & 1) + e] * unit[w];
    }
    __syncthreads();
#pragma unroll 1
    for (int m = lane / span; m < 16; m += 64 / span) {
      if (16 * i + m >= t.rows || n0 + col >= outputs) continue;
      const int swap = 32 * ((m >> 2) & 1);
      const float v = turn[m * 64 + (col ^ swap)];
      const float up = a.gated ? turn[m * 64 + ((32 + col) ^ swap)] : 0.0f;
      finish(a, t.expert, t.row0 + 16 * i + m, n0 + col, v, up);
    }
    __syncthreads();
  }
}

template <class S>
void go(const LinearArgs& a, const LinearPlan& p, hipStream_t st) {
  const unsigned grid = (unsigned)(p.col_tiles * p.row_tiles);
  if (p.tiles) {
    if (p.blocks == 1) linear_tile_kernel<S, 1><<<grid, 256, 0, st>>>(a, p.col_tiles);
    else if (p.blocks == 2) linear_tile_kernel<S, 2><<<grid, 256, 0, st>>>(a, p.col_tiles);
    else linear_tile_kernel<S, 4><<<grid, 256, 0, st>>>(a, p.col_tiles);
    return;
  }
  const size_t lds = (size_t)p.waves * 2 * p.blocks * 1024;
  if (p.blocks == 1) linear_few_kernel<S, 1, 2><<<grid, 64 * p.waves, lds, st>>>(a, p.col_tiles);
  else if (p.blocks == 2) linear_few_kernel<S, 2, 2><<<grid, 64 * p.waves, lds, st>>>(a, p.col_tiles);
  else linear_few_kernel<S, 4, 2><<<grid, 64 * p.waves, lds, st>>>(a, p.col_tiles);
}

}  // namespace

template <>
hipError_t launch_linear_bits<BITS>(const LinearArgs& a, awq_dtype_t dt, const LinearPlan& p, void*, hipStream_t st) {
  ProfScope prof("awq_lowbit_linear", st);
  if (dt == AWQ_F16) go<_Float16>(a, p, st);
  else go<__bf16>(a, p, st);
  return hipGetLastError();
}

}  // namespace awq
