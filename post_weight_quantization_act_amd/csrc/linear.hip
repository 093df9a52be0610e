// y = act(x W'^T + bias) [times (x W_up'^T + bias_up)] + residual with packed W' = (c - z) step:
// one projection for all rows, or each expert's own for its sorted rows.
//
// The codes' layout is awq_lowbit_repack's: the words of row n's chunk j (32 columns) at
// (j R + n) bits, R the rows of all experts; (step, z) of group g at g R + n.  Codes become the
// exact integers c - z in the activations' type, in the registers that the matrix
// instructions read them from; products are exact and sums are held in fp32, by group, scaled by
// the group's step.  Two kernels: linear_few_kernel for few rows, which waits for the weights alone, and
// linear_tile_kernel, bound by the weights up to some 32 rows an expert and by the matrix
// instructions from some 128 on.
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
  int rows;
  int expert;        // `experts`: rows that no expert here has
};

// Inclusive sums over the wave's lanes.
__device__ __forceinline__ int wave_sums(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // from 1, 2, 4, 8 lanes below in a row of 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // a row's last into the next, a half's into the other
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
  return x;
}

// The rows' tiles of `most` rows, expert by expert, and last those of rows that no expert has.  A lane
// counts a run of experts; of up to 255 it holds their offsets, so that finding a tile waits for
// memory once.
struct Tiles {
  static constexpr int kHeld = 4;
  const LinearArgs& a;
  int most, each, mine, upto, all;     // all: tiles
  int bound[kHeld + 1];

  // Where expert e's rows begin; e = experts: where the others' do.
  __device__ __forceinline__ int begin(int e) const {
    const int total = (int)a.rows, o = e <= a.experts ? a.offsets[e] : total;
    return o < 0 ? 0 : o > total ? total : o;
  }
  __device__ __forceinline__ int tiles_in(int lo, int hi) const { return hi > lo ? (hi - lo + most - 1) / most : 0; }

  __device__ __forceinline__ Tiles(const LinearArgs& args, int most_rows) : a(args), most(most_rows) {
    if (!a.offsets) {
      all = (int)((a.rows + most - 1) / most);
      return;
    }
    each = a.experts / 64 + 1;         // experts + 1 of them in all
    const int e0 = (int)(threadIdx.x & 63) * each;
    mine = 0;
    if (each <= kHeld) {
#pragma unroll
      for (int i = 0; i <= kHeld; ++i) bound[i] = begin(e0 + (i < each ? i : each));
#pragma unroll
      for (int i = 0; i < kHeld; ++i) mine += tiles_in(bound[i], bound[i + 1]);
    } else {
      int lo = begin(e0);
      for (int i = 0; i < each; ++i) {
        const int hi = begin(e0 + i + 1);
        mine += tiles_in(lo, hi);
        lo = hi;
      }
    }
    upto = wave_sums(mine);
    all = __builtin_amdgcn_readlane(upto, 63);
  }
  // Tile want < all.
  __device__ __forceinline__ Tile at(int want) const {
    Tile t;
    if (!a.offsets) {
      t.row0 = (int64_t)want * most;
      const int64_t left = a.rows - t.row0;
      t.rows = (int)(left < most ? left : most);
      t.expert = 0;
      return t;
    }
    const int l = __builtin_ctzll(__ballot(want < upto));
    int lo = 0, hi = 0, e = 0, w = want - (upto - mine);
    if (each <= kHeld) {
      int at = 0;                        // tiles before the run's expert i
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int n = tiles_in(bound[i], bound[i + 1]);
        if (w >= at && w < at + n) {
          e = i;
          lo = bound[i] + (w - at) * most;
          hi = bound[i + 1];
        }
        at += n;
      }
      t.row0 = __builtin_amdgcn_readlane(lo, l);
      hi = __builtin_amdgcn_readlane(hi, l);
      t.expert = l * each + __builtin_amdgcn_readlane(e, l);
    } else {
      w = __builtin_amdgcn_readlane(w, l);
      e = l * each;
      lo = begin(e);
      hi = begin(e + 1);
      for (int n = tiles_in(lo, hi); w >= n && e < a.experts; n = tiles_in(lo, hi)) {
        w -= n;
        ++e;
        lo = hi;
        hi = begin(e + 1);
      }
      t.row0 = lo + w * most;
      t.expert = e;
    }
    t.rows = hi - (int)t.row0 < most ? hi - (int)t.row0 : most;
    return t;
  }
};

// Workgroups are dealt to the eight XCDs in turn.  Each XCD takes a run of tiles, eight row tiles by
// all columns after one another, so that its L2 holds what neighbours share: the activations of
// eight row tiles and an expert's weights.  (The grid is sized by a bound; past the tiles there are
// none.)
struct Place {
  int row, col;
};
__device__ __forceinline__ Place place_of(uint32_t id, uint32_t col_tiles, uint32_t row_tiles) {
  constexpr uint32_t kXcds = 8, kGroup = 8;
  const uint32_t n = col_tiles * row_tiles, per = n / kXcds, more = n % kXcds, x = id % kXcds;
  const uint32_t at = x * per + (x < more ? x : more) + id / kXcds;
  const uint32_t group = at / (kGroup * col_tiles), in = at - group * (kGroup * col_tiles);
  const uint32_t left = row_tiles - group * kGroup, rows = left < kGroup ? left : kGroup;
  return {(int)(group * kGroup + in % rows), (int)(in / rows)};
}

// Row of x that output row r takes.
__device__ __forceinline__ int64_t source(const LinearArgs& a, int64_t r) {
  if (!a.order) return r;
  const int64_t s = (uint32_t)a.order[r] / (uint32_t)a.per_token;
  return s < a.x_rows ? s : 0;
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

// The same in fp16 with fewer instructions, scaled: two codes in the low bits of the halves of a word
// read as the subnormals c 2^-24, and one packed multiply-add makes (c - z) 2^-10 of them, exactly.
// 4 bits: 11 instructions for eight codes, 8 bits: 8, others 16 to 18.
constexpr float kHalfScale = 1024.0f;
template <int P, int NW>
__device__ __forceinline__ uint32_t two_codes(const uint32_t (&w)[NW]) {
  constexpr int b = 2 * BITS * P, wi = b >> 5, o = b & 31;
  if constexpr (BITS == 8) {
    return __builtin_amdgcn_perm(0u, w[wi], o == 0 ? 0x0c010c00u : 0x0c030c02u);
  } else if constexpr (BITS == 4) {
    constexpr uint32_t k = P & 3;
    return __builtin_amdgcn_perm((w[wi] >> 4) & 0x0f0f0f0fu, w[wi] & 0x0f0f0f0fu, 0x0c040c00u + 0x00010001u * k);
  } else {
    constexpr uint32_t field = (1u << 2 * BITS) - 1u, mask = (1u << BITS) - 1u;
    uint32_t p;
    if constexpr (o + 2 * BITS <= 32) p = (w[wi] >> o) & field;
    else p = __builtin_amdgcn_alignbit(w[wi + 1], w[wi], o) & field;
    return (p << (16 - BITS) | p) & (mask | mask << 16);
  }
}
template <int Q, int NW>
__device__ __forceinline__ i32x4 eight_f16(const uint32_t (&w)[NW], bool live, half2v minus) {
  const half2v by = __builtin_bit_cast(half2v, live ? 0x74007400u : 0u);    // 2^14; 0 where a step is 0
  auto one = [&](uint32_t v) {
    return (int)__builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2v, v), by, minus));
  };
  return i32x4{one(two_codes<4 * Q>(w)), one(two_codes<4 * Q + 1>(w)), one(two_codes<4 * Q + 2>(w)),
               one(two_codes<4 * Q + 3>(w))};
}
__device__ __forceinline__ half2v minus_f16(float z) {
  const _Float16 n = (_Float16)(z * (-1.0f / kHalfScale));
  return half2v{n, n};
}

// ---- loads ---------------------------------------------------------------------------------
typedef __amdgpu_buffer_rsrc_t Buffer;

__device__ __forceinline__ Buffer buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
}

// Words at voff + soff bytes: one load for up to four.
template <int NW>
__device__ __forceinline__ void load_words(Buffer b, uint32_t voff, uint32_t soff, uint32_t (&w)[NW]) {
  if constexpr (NW > 4) {
    uint32_t lo[4], hi[NW - 4];
    load_words<4>(b, voff, soff, lo);
    load_words<NW - 4>(b, voff + 16, soff, hi);
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = i < 4 ? lo[i < 4 ? i : 0] : hi[i < 4 ? 0 : i - 4];
  } else if constexpr (NW == 1) {
    w[0] = __builtin_amdgcn_raw_buffer_load_b32(b, voff, soff, 0);
  } else if constexpr (NW == 2) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(b, voff, soff, 0);
    w[0] = v[0], w[1] = v[1];
  } else if constexpr (NW == 3) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b96(b, voff, soff, 0);
    w[0] = v[0], w[1] = v[1], w[2] = v[2];
  } else {
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(b, voff, soff, 0);
    w[0] = v[0], w[1] = v[1], w[2] = v[2], w[3] = v[3];
  }
}

// ---- few rows ---------------------------------------------------------------------------------
// A workgroup takes WT tiles of 16 weight rows (gated: a tile of gates and the same of ups) and
// 16 TT output rows; its waves share the columns of K, 128 at a time, and add up in LDS.  Lane
// 16 g + r holds weight row r and the 32 codes of chunk g of the four: one load of `bits` words;
// instruction i of four multiplies the chunks' codes 8 i .. 8 i + 7.  One row of 8192 to 28672
// columns, 3 bits: 36 us, 2.8 TB/s; bound by unpacking (awq_lowbit_gemv, on the vector units alone, 33; four
// rows 36 and 44; one row of 4096 x 4096, 4 bits, 11 and 13.5, of 11008 to 4096 15 and 14).  8 rows for 8 of 128 experts, 1536 x 2048, 4
// bits: 11 us, of which the weights are 2.7; bound by its chain of loads (offsets, codes, the
// rows' places, the rows).
template <class S, int TT, int WT>
__global__ __launch_bounds__(512, 2) void linear_few_kernel(LinearArgs a, int col_tiles) {
  extern __shared__ __attribute__((aligned(16))) f32x4 red[];      // [waves][WT][TT][64]
  const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int outputs = a.gated ? a.N / 2 : a.N;
  const int wide = a.gated ? 16 : 16 * WT;             // outputs of a workgroup
  const int n0 = (int)(blockIdx.x % (uint32_t)col_tiles) * wide;
  Tiles tiles(a, 16 * TT);
  const uint32_t want = blockIdx.x / (uint32_t)col_tiles;
  if (want >= (uint32_t)tiles.all) return;
  const Tile t = tiles.at(want);
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
  struct Step {
    uint32_t w[WT][BITS];
    float2 m[WT];
    i32x4 x[TT][4];
  };
  auto load_codes = [&](int s, Step& b) __attribute__((always_inline)) {
    const int j = 4 * s + g;
    const int64_t jj = j < chunks ? j : chunks - 1;
#pragma unroll
    for (int w = 0; w < WT; ++w) {
      const uint32_t* p = a.codes + (jj * a.R + wrow[w]) * BITS;
#pragma unroll
      for (int i = 0; i < BITS; ++i) b.w[w][i] = p[i];
      b.m[w] = a.meta[(jj >> a.lg_cpg) * a.R + wrow[w]];
    }
  };
  auto load_x = [&](int s, Step& b) __attribute__((always_inline)) {
    const int64_t j = 4 * s + g;
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        b.x[i][q] = i32x4{0, 0, 0, 0};
        if (x[i] && j < chunks) b.x[i][q] = *(const i32x4*)(x[i] + 32 * j + 8 * q);
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
  // codes before the rows: those wait for their places
  if (s < steps) load_codes(s, cur);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int m = 16 * i + r;
    x[i] = m < t.rows ? (const S*)a.x + source(a, t.row0 + m) * a.stride : nullptr;
  }
  if (s < steps) load_x(s, cur);
  for (; s < steps; s += waves) {
    if (s + waves < steps) load_codes(s + waves, next), load_x(s + waves, next);
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
    float v[1] = {total(a.gated ? 0 : n >> 4, m, n & 15)}, up[1] = {a.gated ? total(WT - 1, m, n) : 0.0f};
    finish(a, t.expert, t.row0 + m, n0 + n, v, up);
  }
}

// ---- many rows -----------------------------------------------------------------------------------
// A workgroup takes 32 MT output rows and 256 weight rows, a wave all the output rows and 64 weight
// rows (gated: 32 gates and the same ups).  Activations go through LDS, 128 columns at a time, two
// buffers; a wave unpacks its own weights in registers, so each code is unpacked once for 32 MT
// rows: lane half h takes codes 16 h .. 16 h + 15 of a chunk.  KS = 2: two sets of four waves take
// every other 128 columns, and add up at the end.
// The sums are in units of the group's step U: where the next group begins they are multiplied by
// U / U', a step of 0 leaves the unit as it is and its codes count as 0.  So what a sum reaches is its
// products by the largest step over the smallest.  (A wave that took sums which left fp32 again, group by
// group, cost every call 7 to 10%: 2047 x 4096 x 11008 185 -> 199 us.)
// WIDE: groups of 128 columns and more, so a step lies in one.
// splits > 1: a workgroup takes the steps of one part of K and leaves fp32 sums to a kernel that joins them.
// 4 bits: 2047 x 4096 x 11008 in fp16 183 us, 1.01 PFLOP/s; 24570 rows for 64 experts, 2816 x 2048, 340
// us, 0.83 PFLOP/s; a library's product of such a size reaches 1.17 to 1.23 here, and this loop by
// itself 1.13.  The rest are rows that the last tile of an expert lacks, and the first loads and last
// stores of a round of workgroups.  488 rows for 128 experts, 1536 x 2048: 55 us, 3.8 TB/s; each step
// waits for its codes, and a ring of three steps in flight gained nothing.
// Workgroups of a compute unit: as many as their registers allow without spills.
constexpr int tile_groups(int mt, bool wide) {
  return mt == 1 ? (BITS <= 4 && wide ? 4 : 3) : mt == 2 && BITS <= 4 && wide ? 3 : 2;
}
template <class S, int MT, int KS, bool WIDE>
__global__ __launch_bounds__(256 * KS, KS == 2 ? 1 : tile_groups(MT, WIDE)) void linear_tile_kernel(LinearArgs a, LinearPlan p) {
  constexpr bool kF16 = sizeof(S) == 2 && std::is_same<S, _Float16>::value;
  constexpr int NW = (BITS + 1) / 2, M = WIDE ? 1 : 4;
  constexpr int kRows = 32 * MT, kPer = 2 * MT;                  // transfers of a wave and step
  constexpr int kPitch = 68;     // floats of a row in the epilogue
  constexpr int kBuffer = kRows * 256, kTurns = KS * 4 * 16 * kPitch * 4;
  __shared__ __attribute__((aligned(1024))) char xs[KS * 2 * kBuffer > kTurns ? KS * 2 * kBuffer : kTurns];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3, set = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 8);
  const int r = lane & 31, h = lane >> 5;
  const int outputs = a.gated ? a.N / 2 : a.N;
  const int wide = a.gated ? 32 : 64;                            // outputs of a wave
  // Two workgroups share a compute unit.  Where more follow, the second of each pair starts 4 us
  // later, so that one multiplies while the other waits for its first rows or stores its last
  // (24570 rows for 64 experts, 2816 x 2048, 4 bits: 362 us without, 337 with 4, 341 with 8; few steps of
  // K: 4096 x 16384 x 128 in fp16 73 us without and 74 with, 256 columns 82 and 83, 512 103 and 103)
  if (MT == 4 && KS == 1 && gridDim.x > 512 && blockIdx.x >= 256 && blockIdx.x < 512)
    for (int i = 0; i < 4; ++i) __builtin_amdgcn_s_sleep(32);
  Tiles tiles(a, kRows);
  const uint32_t part = blockIdx.x % (uint32_t)p.splits, id = blockIdx.x / (uint32_t)p.splits;
  if (id >= (uint32_t)tiles.all * (uint32_t)p.col_tiles) return;
  const Place at = p.splits > 1 ? Place{(int)(id % (uint32_t)tiles.all), (int)(id / (uint32_t)tiles.all)}
                                : place_of(id, p.col_tiles, tiles.all);
  const int first = at.col * 4 * wide, n0 = first + wave * wide;
  const Tile t = tiles.at(at.row);
  if (t.expert == a.experts) {
    const int span = 4 * wide;
    for (int e = tid; e < t.rows * span; e += 256 * KS)
      if (first + e % span < outputs) store_as(a.out, (t.row0 + e / span) * outputs + first + e % span, a.out_type, 0.0f);
    return;
  }
  const int chunks = (int)(a.K / 32), cmask = (1 << a.lg_cpg) - 1, step0 = (int)part * p.per;
  const int steps = step0 + p.per < (chunks + 3) / 4 ? step0 + p.per : (chunks + 3) / 4;    // where this part ends
  const uint32_t R = (uint32_t)a.R;
  uint32_t woff[2], moff[2];
  const int qw = (16 * h * BITS) >> 5, qoff = (16 * h * BITS) & 31;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    int n = n0 + (a.gated ? 0 : 32 * w) + r;
    n = n < outputs ? n : outputs - 1;
    const uint32_t row = (uint32_t)t.expert * a.N + n + (a.gated && w ? outputs : 0);
    woff[w] = (row * BITS + qw) * 4;
    moff[w] = row * 8;
  }
  const Buffer rc = buffer_of(a.codes, (uint32_t)chunks * R * BITS * 4);
  const Buffer rm = buffer_of(a.meta, (uint32_t)(chunks >> a.lg_cpg) * R * 8);
  // activations: transfer q of a step brings rows 4 q .. 4 q + 3, 16-byte part p of row m from
  // part p ^ (m % 16); rows past the last are the first again
  const i32x4 rx = byte_range(a.x, (uint32_t)(((a.x_rows - 1) * a.stride + a.K) * 2));
  const uint32_t base = (uint32_t)(uintptr_t)xs + set * 2 * kBuffer;
  uint32_t xoff[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int m = 4 * (wave * kPer + i) + (lane >> 4);
    const int64_t row = source(a, t.row0 + (m < t.rows ? m : 0));
    xoff[i] = (uint32_t)((row * a.stride + 8 * ((lane & 15) ^ (m & 15))) * 2) + 256 * (step0 + set);
  }
  auto fetch_x = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      to_lds16(rx, base + buf * kBuffer + (wave * kPer + i) * 1024, xoff[i]);
      xoff[i] += 256 * KS;
    }
  };
  struct Codes {
    uint32_t w[2][4][NW];
    float2 m[2][M];
  };
  auto fetch_codes = [&](int s, Codes& c) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      int j = 4 * s + q;
      if (!WIDE) j = j < chunks ? j : chunks - 1;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        load_words<NW>(rc, woff[w], (uint32_t)j * R * (BITS * 4), c.w[w][q]);
        if (q < M) {
          const auto v = __builtin_amdgcn_raw_buffer_load_b64(rm, moff[w], (uint32_t)(j >> a.lg_cpg) * R * 8, 0);
          c.m[w][q < M ? q : 0] = make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
        }
      }
    }
  };
  const QuarterOps<BITS> ops = magic_ops<BITS, QuarterWindows<BITS>::kPer>();
  f32x16 acc[MT][2];
  float unit[2] = {0.0f, 0.0f};      // 0: none yet
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int w = 0; w < 2; ++w) acc[i][w] = f32x16{};
  // where a group begins
  auto rescale = [&](auto blocks, const float2 (&m)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float u = m[w].x != 0.0f ? m[w].x : unit[w], by = unit[w] == 0.0f ? 1.0f : unit[w] / u;   // 1 within a group
#pragma unroll
      for (int i = 0; i < decltype(blocks)::value; ++i) acc[i][w] *= by;
      unit[w] = u;
    }
  };
  typedef i32x4 Weights[2][2];
  auto unpack = [&](const Codes& c, int q, Weights& f) __attribute__((always_inline)) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float2 m = c.m[w][q < M ? q : 0];
      const bool live = m.x != 0.0f;
      uint32_t run[NW];
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        uint32_t v = c.w[w][q][i];
        if constexpr (BITS % 2 == 1) v = i + 1 < NW ? __builtin_amdgcn_alignbit(c.w[w][q][i + 1 < NW ? i + 1 : i], v, qoff) : v >> qoff;
        run[i] = kF16 || live ? v : 0u;
      }
      const float z = live ? m.y : 0.0f;
      if constexpr (kF16) {
        const half2v minus = minus_f16(z);
        f[w][0] = eight_f16<0>(run, live, minus);
        f[w][1] = eight_f16<1>(run, live, minus);
      } else {
        const Zero zero(z);
        f[w][0] = eight<S, NW, 0>(run, zero.neg, zero.sub, ops);
        f[w][1] = eight<S, NW, 1>(run, zero.neg, zero.sub, ops);
      }
    }
  };
  auto multiply = [&](auto blocks, int s, const Codes& c, const char* xb) __attribute__((always_inline)) {
    constexpr int B = decltype(blocks)::value;      // row blocks that there are
    if (WIDE) rescale(blocks, {c.m[0][0], c.m[1][0]});
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = 4 * s + q;
      if (!WIDE) {
        if (j >= chunks) break;
        if ((j & cmask) == 0 || q == 0) rescale(blocks, {c.m[0][q < M ? q : 0], c.m[1][q < M ? q : 0]});
      }
      Weights f;
      unpack(c, q, f);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const int m = 32 * i + r, p = 4 * q + 2 * h + k;
          const i32x4 fa = *(const i32x4*)(xb + m * 256 + 16 * (p ^ (m & 15)));
#pragma unroll
          for (int w = 0; w < 2; ++w) acc[i][w] = mfma32<S>(fa, f[w][k], acc[i][w]);
        }
    }
  };
  auto run = [&](auto blocks) __attribute__((always_inline)) {
    Codes one, two;
    auto step = [&](int s, Codes& cur, Codes& next, int buf) __attribute__((always_inline)) {
      if (s + KS < steps) {
        fetch_x(buf ^ 1);
        fetch_codes(s + KS, next);
      }
      if (s < steps) multiply(blocks, s, cur, xs + (set * 2 + buf) * kBuffer);
      vm_wait<0>();
      __syncthreads();
    };
    if (step0 + set < steps) {
      fetch_x(0);
      fetch_codes(step0 + set, one);
    }
    vm_wait<0>();
    __syncthreads();
    for (int s = step0; s < steps; s += 2 * KS) {
      step(s + set, one, two, 0);
      if (s + KS < steps) step(s + KS + set, two, one, 1);
    }
  };
  // an expert's last tile of half the rows or fewer takes half the products
  if (MT > 1 && t.rows <= 16 * MT) {
    asm volatile("");
    run(std::integral_constant<int, (MT + 1) / 2>());
  } else {
    run(std::integral_constant<int, MT>());
  }
  // Lane l holds weight row l % 32 and output rows 8 (e / 4) + 4 (l / 32) + e % 4.  Sixteen rows at
  // a time go through LDS, from where a lane takes four columns of a row: 16 lanes a row (gated: 8).
  float* turn = (float*)xs + wave * 16 * kPitch;
  const int span = a.gated ? 8 : 16, col = 4 * (lane % span);
  // a wave's LDS operations are in order; two sets wait for each other
  auto meet = [&]() __attribute__((always_inline)) {
    if (KS == 2) __syncthreads();
    else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
#pragma unroll
  for (int w = 0; w < 2; ++w) unit[w] *= !kF16 ? 1.0f : a.x_scale ? kHalfScale / (1 << kRowScale) : kHalfScale;
#pragma unroll 1
  for (int i = 0; i < 2 * MT && 16 * i < t.rows; ++i) {
#pragma unroll
    for (int k = 0; k < 2 * MT; ++k) {
      if (k != i) continue;              // registers have no index: a copy of the stores for each, one of the rest
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int m = 8 * (e >> 2) + 4 * h + (e & 3);
#pragma unroll
        for (int w = 0; w < 2; ++w)
          turn[set * (4 * 16 * kPitch) + m * kPitch + 32 * w + r] = acc[k >> 1][w][8 * (k & 1) + e] * unit[w];
      }
    }
    meet();
#pragma unroll 1
    for (int m = lane / span + set * (64 / span); m < 16; m += 64 / span * KS) {
      if (16 * i + m >= t.rows) continue;
      f32x4 v = *(const f32x4*)&turn[m * kPitch + col], up = *(const f32x4*)&turn[m * kPitch + 32 + col % 32];
      if (KS == 2) {
        v += *(const f32x4*)&turn[4 * 16 * kPitch + m * kPitch + col];
        up += *(const f32x4*)&turn[4 * 16 * kPitch + m * kPitch + 32 + col % 32];
      }
      const int64_t row = t.row0 + 16 * i + m;
      if (a.x_scale) {
        const float by = a.x_scale[source(a, row)];
        v *= by;
        up *= by;
      }
      if (p.splits > 1) {
        float* to = p.partial + ((int64_t)part * a.rows + row) * a.N + n0 + col;
        if (n0 + col + 4 <= outputs) {
          const float x[4] = {v[0], v[1], v[2], v[3]}, y[4] = {up[0], up[1], up[2], up[3]};
          store_run<4>(to, x);
          if (a.gated) store_run<4>(to + outputs, y);
        } else {
          for (int c = 0; c < outputs - n0 - col; ++c) {
            to[c] = c == 0 ? v[0] : c == 1 ? v[1] : v[2];
            if (a.gated) to[outputs + c] = c == 0 ? up[0] : c == 1 ? up[1] : up[2];
          }
        }
      } else if (n0 + col + 4 <= outputs) {
        float x[4] = {v[0], v[1], v[2], v[3]}, y[4] = {up[0], up[1], up[2], up[3]};
        finish(a, t.expert, row, n0 + col, x, y);
      } else {
        for (int c = 0; c < outputs - n0 - col; ++c) {
          float x[1] = {c == 0 ? v[0] : c == 1 ? v[1] : v[2]}, y[1] = {c == 0 ? up[0] : c == 1 ? up[1] : up[2]};
          finish(a, t.expert, row, n0 + col + c, x, y);
        }
      }
    }
    meet();
  }
}

template <class S, int KS, bool WIDE>
void go_tiles(const LinearArgs& a, const LinearPlan& p, unsigned grid, hipStream_t st) {
  grid *= p.splits;
  if (p.blocks == 1) linear_tile_kernel<S, 1, KS, WIDE><<<grid, 256 * KS, 0, st>>>(a, p);
  else if (p.blocks == 2) linear_tile_kernel<S, 2, KS, WIDE><<<grid, 256 * KS, 0, st>>>(a, p);
  else linear_tile_kernel<S, 4, KS, WIDE><<<grid, 256 * KS, 0, st>>>(a, p);
}
template <class S, bool WIDE>
void go_sets(const LinearArgs& a, const LinearPlan& p, unsigned grid, hipStream_t st) {
  if (p.waves == 8) go_tiles<S, 2, WIDE>(a, p, grid, st);
  else go_tiles<S, 1, WIDE>(a, p, grid, st);
}

template <class S>
void go(const LinearArgs& a, const LinearPlan& p, hipStream_t st) {
  const unsigned grid = (unsigned)(p.col_tiles * p.row_tiles);
  if (p.tiles) {
    if (a.lg_cpg >= 2) go_sets<S, true>(a, p, grid, st);
    else go_sets<S, false>(a, p, grid, st);
    return;
  }
  const size_t lds = (size_t)p.waves * 2 * p.blocks * 1024;
  if (p.blocks == 1) linear_few_kernel<S, 1, 2><<<grid, 64 * p.waves, lds, st>>>(a, p.col_tiles);
  else linear_few_kernel<S, 2, 2><<<grid, 64 * p.waves, lds, st>>>(a, p.col_tiles);
}

}  // namespace

template <>
hipError_t launch_linear_bits<BITS>(const LinearArgs& a, awq_dtype_t dt, const LinearPlan& p, hipStream_t st) {
  ProfScope prof("awq_lowbit_linear", st);
  if (dt == AWQ_F16) go<_Float16>(a, p, st);
  else go<__bf16>(a, p, st);
  return hipGetLastError();
}

}  // namespace awq
