// Attention over the paged 8-bit cache.
//
//   o = sum_j p_j v_j,  p = softmax_j(scale q . k_j)  over the tokens j that the row sees,
//   k_j = (u - 128) step of its page and head, v_j likewise.
// A row that sees nothing gives 0, and -inf for the logarithm of its sum.
//
// One pass over the cache.  A wave takes tiles of 64 tokens and tiles of 16 rows
// (rows: the query heads that share a kv head, token after token) and stays in
// registers: S^T = K Q^T leaves each lane 16 scores of one row, in the order in
// which O^T += V^T P^T wants its probabilities, because the rows of the K tiles
// are taken in the order token(i, m) = 16 (m / 4) + 4 i + m % 4 (tile i of 4, row m
// of 16): lane 16 g + q then holds tokens 16 g .. 16 g + 15 of row q.  A page holds a
// multiple of 16 tokens, so those sixteen share one page, one key step and one
// value step.
//
// Codes become fp16 exactly: the byte u under 0x64 reads 1024 + u, and a packed
// subtraction of 1152 leaves u - 128.  (Scores could keep the surplus and subtract 1152
// sum_d q_d at the end: 64 instructions fewer a tile, no faster where memory bounds
// the kernel, and ten times the rounding, which shows in the lse of short rows.)
// Queries are scaled by a power of two of their row to |q| < 2 and are exact in fp16
// but for bf16 elements more than 2^-14 below their row's largest, which keep 24 bits
// below 1.
//
// With t = log2 of (weight times value step), one reference R for each row serves
// sums and values: p = exp2(t - R) weighs the codes, and the row's sum adds
// p / step once for sixteen tokens, in fp32.  p is rounded to fp16 for the matrix
// cores; R follows the largest t so that p stays below 2^15 and above 2^-14 with
// full precision for everything within 2^-22 of the row's largest contribution.
//
// attention_kernel: few rows.  Bound by memory where the cache is long: one sequence of
// 131071 tokens, 64 heads over 8, 52 us (5.2 TB/s, cold) and 5 us to join; by the latency of a
// tile (2.3 us a wave: values, scores, exponentials, values' product) where sequences are
// short or uneven: 64 of 1 to 8192 tokens 33 + 5 us; one of 513 tokens, 32 heads 8.5 us.
// attention_rows_kernel: many rows, bound by neither unit alone: 2 x 2047 rows of 64 heads
// over 3000 and 4096 tokens 460 to 466 us, 727 to 736 TFLOP/s (a large fp16 matrix product
// reaches 1140 to 1180 here); the matrix units are busy 29% and the vector units 50% of the
// time, 1.5 waves a SIMD on average.
#include <algorithm>

#include "kv.h"

namespace awq {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr int kTile = 64;                 // tokens of a wave's tile
constexpr float kTop = 15.0f, kRest = 8.0f;   // R follows when t - R passes kTop, to t - kRest
constexpr float kLeastFactor = 1e-30f;
constexpr float kLeastStep = 7.888609052210118e-31f;   // 2^-100: a value step below counts as 0

struct Split {
  int splits;        // workgroups along the tokens of one row tile
  int tiles;         // 64-token tiles of each; where `chosen` is set, the least, a power of two
  int row_tiles;     // row tiles of a sequence and kv head
  int slots;         // workgroups that run at once
  float* o;          // [splits][T * Hq][D], null when splits == 1
  float2* rl;        // [splits][T * Hq]: reference and sum
  int* chosen;       // where the first kernel tells the second what it took for `tiles`; or null
};

constexpr int kChoices = 5;

// Rows of a sequence's n that the call takes: the first ones.
__device__ __forceinline__ int taken(const AttArgs& a, int n) { return n < a.max_new ? n : a.max_new; }

// 64-token tiles that the rows of a sequence see, so at least as many as any of its row
// tiles does; -1: it has no rows.
__device__ __forceinline__ int tiles_of(const AttArgs& a, int b) {
  int64_t row0;
  int n, lo, hi, unused;
  rows_of(a.c, b, row0, n);
  if (n == 0) return -1;
  seen_by(a, a.lens[b], n, 0, lo, unused);
  seen_by(a, a.lens[b], n, taken(a, n) - 1, unused, hi);
  return hi > lo ? (hi + kTile - 1) / kTile - lo / kTile : 0;
}

__device__ __forceinline__ int splits_of(int nt, int tiles_log) {
  return nt > 0 ? ((nt - 1) >> tiles_log) + 1 : nt + 1;
}

// Sequences differ in length and the host does not know them: every workgroup looks at
// all lengths (at most one a thread), takes for the tiles of a split the least power of
// two times sp.tiles for which all splits run at once, or that is twice a slot's share
// of all tiles, and finds its own split by counting: no workgroup but the last few is
// empty.  (A grid of sequences x most splits costs about a microsecond for every 512
// empty ones: registers let only two at a time onto a compute unit.)  64 sequences of
// 1 to 8192 tokens, 8 heads: 32 to 35 us; it was 29, against 33 with a fixed 20 tiles a
// split, before the keys were centred.
struct Part {
  int tiles, b, split;    // b = -1: nothing is left for this workgroup
};

template <int THREADS>
__device__ __forceinline__ Part choose(const AttArgs& a, const Split& sp, int want) {
  constexpr int W = THREADS / 64;
  __shared__ int sums[W][kChoices + 1], scan[W], found[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int log = 31 - __builtin_clz(sp.tiles);
  const int nt = tid < a.c.B ? tiles_of(a, tid) : -1;
  int count[kChoices], all = nt > 0 ? nt : 0;
#pragma unroll
  for (int k = 0; k < kChoices; ++k) count[k] = splits_of(nt, log + k);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    all += __shfl_xor(all, m);
#pragma unroll
    for (int k = 0; k < kChoices; ++k) count[k] += __shfl_xor(count[k], m);
  }
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < kChoices; ++k) sums[wave][k] = count[k];
    sums[wave][kChoices] = all;
  }
  if (tid == 0) found[0] = -1;
  __syncthreads();
  int64_t total = 0;    // a wave's 64 sequences have at most 2^30 tiles
  for (int w = 0; w < W; ++w) total += sums[w][kChoices];
  const int64_t groups = (int64_t)a.c.Hkv * sp.row_tiles;
  int take = log;
#pragma unroll
  for (int k = 0; k < kChoices; ++k) {
    int units = 0;
    for (int w = 0; w < W; ++w) units += sums[w][k];
    take = log + k;
    if (units * groups <= sp.slots || ((int64_t)sp.slots << take) >= 2 * total * groups) break;
  }
  const int mine = splits_of(nt, take);
  int upto = mine;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int x = __shfl_up(upto, m);
    upto += lane >= m ? x : 0;
  }
  if (lane == 63) scan[wave] = upto;
  __syncthreads();
  for (int w = 0; w < W; ++w) upto += w < wave ? scan[w] : 0;
  const int at = want - (upto - mine);
  if (at >= 0 && at < mine) {
    found[0] = tid;
    found[1] = at;
  }
  __syncthreads();
  return {1 << __builtin_amdgcn_readfirstlane(take), __builtin_amdgcn_readfirstlane(found[0]),
          __builtin_amdgcn_readfirstlane(found[1])};
}

__device__ __forceinline__ float xor_max(float x) {   // over the four lane groups
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

__device__ __forceinline__ float xor_sum(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Eight codes as fp16 values u - 128.
__device__ __forceinline__ half8 centred(uint32_t lo, uint32_t hi) {
  struct { uint32_t v[4]; } r;
  r.v[0] = __builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u);
  r.v[1] = __builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u);
  r.v[2] = __builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u);
  r.v[3] = __builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u);
  const half8 less = {1152, 1152, 1152, 1152, 1152, 1152, 1152, 1152};
  return __builtin_bit_cast(half8, r) - less;
}

// One row tile's queries, bounds and running state.
template <int DB>
struct Rows {
  half8 q[DB];       // 8 columns of each 32-block
  float f;           // scale log2(e) 2^e of the row
  int lo, hi;        // tokens that the row sees
  float r, l;        // reference, this lane's share of the sum
  f32x4 o[2 * DB];   // O^T: columns 16 dt + 4 g + i
};

// Rows of a tile: the column that MFMA step ks of lane group g starts at.
template <bool W16>
__device__ __forceinline__ int column(int ks, int g) {
  return W16 ? 64 * (ks >> 1) + 16 * g + 8 * (ks & 1) : 32 * ks + 8 * g;
}

template <class T, int DB, bool W16>
__device__ __forceinline__ void load_rows(const AttArgs& a, Rows<DB>& w, int64_t row0, int n, int len,
                                          int h, int rr, int g) {
  typedef typename T::storage S;
  const int G = a.Hq / a.c.Hkv, i = rr / G;
  w.r = -INFINITY;
  w.l = 0.0f;
  w.lo = 0;
  w.hi = INT32_MAX;   // a row that is not there sees everything: it masks no tile
#pragma unroll
  for (int dt = 0; dt < 2 * DB; ++dt) w.o[dt] = f32x4{0, 0, 0, 0};
  float x[DB][8];
  const bool valid = i < taken(a, n);
  if (valid) seen_by(a, len, n, i, w.lo, w.hi);
  if (w.lo == w.hi) w.lo = w.hi = 0;   // before every token, so that no block's steps count
  const S* q = (const S*)a.q + (row0 + (valid ? i : 0)) * a.qs[0] + (h * G + (valid ? rr % G : 0)) * a.qs[1];
  uint32_t top = 0;
#pragma unroll
  for (int ks = 0; ks < DB; ++ks) {
    const int d = column<W16>(ks, g);
    struct V { S v[8]; } v;
    const bool in = valid && d < a.c.D;
    v = in ? __builtin_bit_cast(V, *(const u32x4_loose*)(q + d)) : V{};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[ks][j] = to_f32(v.v[j]);
      const uint32_t m = abs_bits(x[ks][j]);
      top = top > m ? top : m;
    }
  }
  // the row's largest exponent, from all four groups (orders like the values for these bits)
  float m = xor_max(__uint_as_float(top > 0x7f7fffffu ? 0x3f800000u : top));
  int e = (int)(__float_as_uint(m) >> 23) - 127;
  e = m == 0.0f ? 0 : e;
#pragma unroll
  for (int ks = 0; ks < DB; ++ks)
#pragma unroll
    for (int j = 0; j < 8; ++j) w.q[ks][j] = (_Float16)ldexpf(x[ks][j], -e);
  w.f = ldexpf(a.scale * kLog2e, e);
}

// The steps of a lane's sixteen tokens.  One that is not finite is NaN for everything
// that its block touches.
struct Steps {
  float ks, log_sv, inv_sv;
  bool zero, there;    // a value step of 0 weighs in the sum and adds nothing

  __device__ __forceinline__ Steps(float k, float v, bool page) {
    ks = k + (k - k);
    v += v - v;
    zero = v < kLeastStep;
    v = zero ? kLeastStep : v;
    log_sv = __builtin_amdgcn_logf(v);
    inv_sv = __builtin_amdgcn_rcpf(v);
    there = page;
  }
};

// Scores of a row tile to probabilities: lane 16 g + q holds row q and tokens tok ..
// tok + 15, score 4 i + j of them in s[i][j].  The reference follows the largest and
// takes what has been summed with it.
template <int DB>
__device__ __forceinline__ void probabilities(Rows<DB>& r, f32x4 (&s)[4], half8 (&p)[2],
                                              const Steps& st, int tok) {
  // a row that sees none of the lane's tokens takes nothing from their block, NaN or not
  const bool some = st.there && r.lo < tok + 16 && tok < r.hi;
  const bool whole = st.there && r.lo <= tok && tok + 16 <= r.hi;
  const float f = some ? r.f * st.ks : 1.0f, lg = some ? st.log_sv : 0.0f;
  if (__any(!whole)) {
    const uint32_t from = (uint32_t)(tok - r.lo), span = some ? (uint32_t)(r.hi - r.lo) : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] = from + (uint32_t)(4 * i + j) < span ? s[i][j] : -INFINITY;
  }
  float top = s[0][0];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) top = fmaxf(top, s[i][j]);
  // a factor of 0 would make NaN of the -inf of tokens that are not seen
  const float fp = f < kLeastFactor ? kLeastFactor : f;
  top = xor_max(fmaf(top, fp, lg));
  if (__any(top > r.r + kTop)) {
    const float to = top > r.r + kTop ? top - kRest : r.r;
    const float by = to == r.r ? 1.0f : __builtin_amdgcn_exp2f(r.r - to);
    r.r = to;
    r.l *= by;
#pragma unroll
    for (int dt = 0; dt < 2 * DB; ++dt) r.o[dt] *= by;
  }
  const float off = lg - (r.r == -INFINITY ? 0.0f : r.r);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float e = __builtin_amdgcn_exp2f(fmaf(s[i][j], fp, off));
      sum += e;
      p[i >> 1][4 * (i & 1) + j] = (_Float16)e;
    }
  if (__any(st.zero)) {
    asm volatile("");    // a branch, and not sixteen selects
    p[0] = st.zero ? half8{} : p[0];
    p[1] = st.zero ? half8{} : p[1];
  }
  r.l += some ? sum * st.inv_sv : 0.0f;
}

// The codes and steps of one 64-token tile on their way in.
template <int DB>
struct Keys {
  u32x4 k[4][(DB + 1) / 2];
  float ks, sv;
  bool there;        // the lane's sixteen tokens have a page
};

// Where a lane finds its keys (rows 16 (c / 4) + 4 i + c % 4 of a tile) and its values and
// steps (tokens 16 g .. 16 g + 15).
struct Finder {
  const uint8_t *k, *v;          // of page 0
  const float *ks, *vs;
  const int32_t* row;            // the sequence's page table
  uint32_t page_bytes, heads, n_pages;
  int last, shift, mask, k_tok, v_tok, D, P;

  __device__ __forceinline__ Finder(const KvArgs& c, int b, int h, int lane) {
    const int col = lane & 15, g = lane >> 4;
    row = c.pages + (int64_t)b * c.max_pages;
    last = c.max_pages - 1;
    shift = c.p_shift;
    mask = c.P - 1;
    n_pages = (uint32_t)c.n_pages;
    heads = (uint32_t)c.Hkv;
    page_bytes = (uint32_t)c.Hkv * (uint32_t)c.P * (uint32_t)c.D;   // below 2^31
    D = c.D;
    P = c.P;
    k_tok = 16 * (col >> 2);
    v_tok = 16 * g;
    k = c.k_codes + (uint32_t)h * c.P * c.D;
    v = c.v_codes + (uint32_t)h * c.P * c.D;
    ks = c.k_steps + h;
    vs = c.v_steps + h;
  }
  __device__ __forceinline__ int page(int tile, int tok) const { return (tile * kTile + tok) >> shift; }
  // Entries for a tile, inside the table; used a tile later, when they have come.
  __device__ __forceinline__ int2 entries(int tile) const {
    const int pk = page(tile, k_tok), pv = page(tile, v_tok);
    return make_int2(row[pk < last ? pk : last], row[pv < last ? pv : last]);
  }
  __device__ __forceinline__ bool there(int entry, int tile, int tok) const {
    return page(tile, tok) <= last && (uint32_t)entry < n_pages;
  }
  // Pointers into the tile; a page that is not there reads as page 0 and is masked.
  __device__ __forceinline__ const uint8_t* keys(int2 e, int tile, int col) const {
    const uint32_t id = there(e.x, tile, k_tok) ? (uint32_t)e.x : 0u;
    return k + (uint64_t)id * page_bytes + (uint32_t)(((tile * kTile + k_tok + (col & 3)) & mask) * D);
  }
  __device__ __forceinline__ const uint8_t* values(int2 e, int tile) const {
    const uint32_t id = there(e.y, tile, v_tok) ? (uint32_t)e.y : 0u;
    return v + (uint64_t)id * page_bytes + (uint32_t)((tile * kTile + v_tok) & mask);
  }
  __device__ __forceinline__ uint64_t block(int2 e, int tile) const {
    return (uint64_t)(there(e.y, tile, v_tok) ? (uint32_t)e.y : 0u) * heads;
  }
};

template <int DB, bool W16>
__device__ __forceinline__ void load_keys(const Finder& f, Keys<DB>& k, int2 e, int tile, int lane) {
  const int col = lane & 15, g = lane >> 4, D = f.D;
  const uint8_t* p = f.keys(e, tile, col);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* r = p + 4 * i * D;
    if (W16) {
#pragma unroll
      for (int s = 0; s < DB / 2; ++s) k.k[i][s] = *(const u32x4*)(r + 64 * s + 16 * g);
    } else {
#pragma unroll
      for (int s = 0; s < DB; ++s) {
        const int d = column<false>(s, g);
        const u32x2 v = *(const u32x2*)(r + (d < D ? d : 0));   // past the head: times a query of 0
        k.k[i][s >> 1][2 * (s & 1)] = v[0];
        k.k[i][s >> 1][2 * (s & 1) + 1] = v[1];
      }
    }
  }
  const uint64_t blk = f.block(e, tile);
  k.there = f.there(e.y, tile, f.v_tok);
  k.ks = f.ks[blk];
  k.sv = f.vs[blk];
}

// NW waves share the tokens of one row tile (QT x 16 rows) and split; their
// results meet in LDS.
template <class T, int DB, int QT, int NW, bool W16>
__global__ __launch_bounds__(NW * 64, DB <= 6 ? 2 : 1) void attention_kernel(AttArgs a, Split sp) {
  typedef typename T::storage S;
  constexpr int DT = 2 * DB;
  constexpr int kPitch = 32 * DB + 4;
  __shared__ __attribute__((aligned(16))) float so[NW][QT * 16][kPitch];
  __shared__ float2 srl[NW][QT * 16];
  const KvArgs& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;

  // heads first, splits last: workgroups are dealt to the eight XCDs in turn, so a
  // sequence's splits, of which only the first few may hold tokens, never fall on one
  // XCD, and with 8 heads the row tiles of a head read its keys through one L2
  uint32_t bid = a.first_block + blockIdx.x;
  int b, rt, split;
  const int h = (int)(bid % (uint32_t)c.Hkv);
  bid /= (uint32_t)c.Hkv;
  if (sp.chosen) {
    rt = (int)(bid % (uint32_t)sp.row_tiles);
    const Part u = choose<NW * 64>(a, sp, (int)(bid / (uint32_t)sp.row_tiles));
    if (a.first_block + blockIdx.x == 0 && tid == 0) *sp.chosen = u.tiles;
    if (u.b < 0) return;
    sp.tiles = u.tiles;
    b = u.b;
    split = u.split;
  } else {
    b = (int)(bid % (uint32_t)c.B);
    bid /= (uint32_t)c.B;
    rt = (int)(bid % (uint32_t)sp.row_tiles);
    split = (int)(bid / (uint32_t)sp.row_tiles);
  }
  int64_t row0;
  int n;
  rows_of(c, b, row0, n);
  const int G = a.Hq / c.Hkv, base = rt * 16 * QT, rows = taken(a, n) * G;
  if (base >= rows) return;
  const int len = a.lens[b];
  int lo, hi, unused;
  seen_by(a, len, n, base / G, lo, unused);
  seen_by(a, len, n, (base + 16 * QT < rows ? base + 16 * QT - 1 : rows - 1) / G, unused, hi);
  const int t0 = lo / kTile, nt = hi > lo ? (hi + kTile - 1) / kTile - t0 : 0;
  const int s0 = t0 + split * sp.tiles;
  const int s1 = s0 + sp.tiles < t0 + nt ? s0 + sp.tiles : t0 + nt;
  if (split > 0 && s0 >= s1) return;
  const bool alone = nt <= sp.tiles;    // no other split has tokens of these rows

  Rows<DB> w[QT];
#pragma unroll
  for (int qt = 0; qt < QT; ++qt)
    load_rows<T, DB, W16>(a, w[qt], row0, n, len, h, base + 16 * qt + col, g);

  Keys<DB> kt;
  const Finder find(c, b, h, lane);
  int2 id = make_int2(0, 0), next = id;
  int tile = s0 + wave;
  if (tile < s1) {
    id = find.entries(tile);
    next = find.entries(tile + NW);
    load_keys<DB, W16>(find, kt, id, tile, lane);
  }
  for (; tile < s1; tile += NW) {
    // values of this tile: sixteen tokens of column 16 dt + col
    u32x4 v[DT];
    {
      const uint8_t* p = find.values(id, tile);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        const int d = 16 * dt + col;
        v[dt] = *(const u32x4*)(p + (d < c.D ? d : 0) * c.P);
      }
    }
    f32x4 s[QT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) s[qt][i] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int ks = 0; ks < DB; ++ks) {
        const u32x4 raw = kt.k[i][ks >> 1];
        const half8 k8 = centred(raw[2 * (ks & 1)], raw[2 * (ks & 1) + 1]);
#pragma unroll
        for (int qt = 0; qt < QT; ++qt)
          s[qt][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k8, w[qt].q[ks], s[qt][i], 0, 0, 0);
      }
    }
    const Steps st(kt.ks, kt.sv, kt.there);
    const int tok = tile * kTile + 16 * g;
    if (tile + NW < s1) {
      id = next;
      load_keys<DB, W16>(find, kt, id, tile + NW, lane);
      next = find.entries(tile + 2 * NW);
    }
    half8 p[QT][2];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) probabilities<DB>(w[qt], s[qt], p[qt], st, tok);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const half8 v0 = centred(v[dt][0], v[dt][1]), v1 = centred(v[dt][2], v[dt][3]);
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) {
        w[qt].o[dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p[qt][0], w[qt].o[dt], 0, 0, 0);
        w[qt].o[dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p[qt][1], w[qt].o[dt], 0, 0, 0);
      }
    }
  }

  // the waves' results meet
#pragma unroll
  for (int qt = 0; qt < QT; ++qt) {
    const float l = xor_sum(w[qt].l);
    if (g == 0) srl[wave][16 * qt + col] = make_float2(w[qt].r, l);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) *(f32x4*)&so[wave][16 * qt + col][16 * dt + 4 * g] = w[qt].o[dt];
  }
  __syncthreads();
  const int quads = c.D / 4;
  for (int e = tid; e < 16 * QT * quads; e += NW * 64) {
    const int r = e / quads, d = 4 * (e % quads), rr = base + r;
    if (rr >= rows) break;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < NW; ++k) top = fmaxf(top, srl[k][r].x);
    f32x4 o = {0, 0, 0, 0};
    float l = 0.0f;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float2 x = srl[k][r];
      const float by = x.x == top ? 1.0f : __builtin_amdgcn_exp2f(x.x - top);
      o += *(const f32x4*)&so[k][r][d] * by;
      l += x.y * by;
    }
    const int64_t out = (row0 + rr / G) * a.Hq + h * G + rr % G;
    if (alone) {
      const float by = l == 0.0f ? 0.0f : 1.0f / l;
      struct { S v[4]; } y;
#pragma unroll
      for (int j = 0; j < 4; ++j) y.v[j] = from_f32<S>(o[j] * by);
      *(u32x2*)((S*)a.out + out * c.D + d) = __builtin_bit_cast(u32x2, y);
      if (d == 0 && a.lse) a.lse[out] = l == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(l)) * kLn2;
    } else {
      const int64_t part = split * c.T * a.Hq + out;
      *(f32x4*)(sp.o + part * c.D + d) = o;
      if (d == 0) sp.rl[part] = make_float2(top, l);
    }
  }
}

// The order of a block of N fragment reads that feed M matrix instructions each: four
// reads ahead of their use (left alone, the compiler waits for each just before it;
// 128 columns 470 -> 455 us for 2 x 2047 rows, eight ahead 463).  Narrow heads, whose
// registers let three workgroups onto a compute unit, are 1% faster without.
template <int N, int M>
__device__ __forceinline__ void reads_ahead() {
  constexpr int kAhead = N < 4 ? N : 4;
  __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
  for (int i = 0; i < N - kAhead; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, M, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, M * kAhead, 0);
}

// Many rows: NW waves of 32 rows each share every tile, which is turned into fp16
// fragments in LDS once for all of them; two buffers and one barrier a tile.  Each wave
// fetches its part of the codes a tile ahead into registers.
template <class T, int DB, int NW, bool W16>
__global__ __launch_bounds__(NW * 64, DB > 4 ? 1 : 2) void attention_rows_kernel(AttArgs a, Split sp) {
  typedef typename T::storage S;
  constexpr int QT = 2, DT = 2 * DB;
  constexpr int KU = W16 ? 2 * DB : 4 * DB;                     // parts of a tile's keys: 1 KB or 512 bytes each
  constexpr int KN = (KU + NW - 1) / NW, VN = (DT + NW - 1) / NW;   // parts of a wave
  __shared__ half8 kf[2][4 * DB][64], vf[2][2 * DT][64];
  const KvArgs& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;

  uint32_t bid = a.first_block + blockIdx.x;
  const int h = (int)(bid % (uint32_t)c.Hkv);
  bid /= (uint32_t)c.Hkv;
  const int b = (int)(bid % (uint32_t)c.B);
  bid /= (uint32_t)c.B;
  const int split = (int)(bid / (uint32_t)sp.row_tiles);
  const int rt = sp.row_tiles - 1 - (int)(bid % (uint32_t)sp.row_tiles);   // the longest first
  int64_t row0;
  int n;
  rows_of(c, b, row0, n);
  const int G = a.Hq / c.Hkv, base = rt * 32 * NW, rows = taken(a, n) * G;
  if (base >= rows) return;
  const int len = a.lens[b];
  int lo, hi, unused;
  seen_by(a, len, n, base / G, lo, unused);
  seen_by(a, len, n, (base + 32 * NW < rows ? base + 32 * NW - 1 : rows - 1) / G, unused, hi);
  const int t0 = lo / kTile, nt = hi > lo ? (hi + kTile - 1) / kTile - t0 : 0;
  const int s0 = t0 + split * sp.tiles;
  const int s1 = s0 + sp.tiles < t0 + nt ? s0 + sp.tiles : t0 + nt;
  if (split > 0 && s0 >= s1) return;
  const bool alone = nt <= sp.tiles;
  const int mine = base + 32 * wave;     // this wave's first row, and the tokens that its rows see
  int w_lo = 0, w_hi = 0;
  if (mine < rows) {
    seen_by(a, len, n, mine / G, w_lo, unused);
    seen_by(a, len, n, (mine + 32 < rows ? mine + 31 : rows - 1) / G, unused, w_hi);
  }

  Rows<DB> w[QT];
#pragma unroll
  for (int qt = 0; qt < QT; ++qt)
    load_rows<T, DB, W16>(a, w[qt], row0, n, len, h, mine + 16 * qt + col, g);

  u32x4 kr[KN], vr[VN];
  float ks = 0.0f, sv = 0.0f, next_ks = 0.0f, next_sv = 0.0f;
  bool there = false, next_there = false;
  const Finder find(c, b, h, lane);
  int2 entry = make_int2(0, 0);       // of the tile after the one that is on its way
  auto fetch = [&](int tile) {
    const int2 e = entry;
    entry = find.entries(tile + 1);
    const uint8_t *kp = find.keys(e, tile, col), *vp = find.values(e, tile);
#pragma unroll
    for (int k = 0; k < KN; ++k) {
      const int u = wave + k * NW;
      if (KU % NW != 0 && u >= KU) break;
      if (W16) {
        kr[k] = *(const u32x4*)(kp + 4 * (u / (DB / 2)) * c.D + 64 * (u % (DB / 2)) + 16 * g);
      } else {
        const int d = column<false>(u % DB, g);
        const u32x2 x = *(const u32x2*)(kp + 4 * (u / DB) * c.D + (d < c.D ? d : 0));
        kr[k][0] = x[0];
        kr[k][1] = x[1];
      }
    }
#pragma unroll
    for (int k = 0; k < VN; ++k) {
      const int dt = wave + k * NW, d = 16 * dt + col;
      if (DT % NW != 0 && dt >= DT) break;
      vr[k] = *(const u32x4*)(vp + (d < c.D ? d : 0) * c.P);
    }
    const uint64_t blk = find.block(e, tile);
    next_ks = find.ks[blk];
    next_sv = find.vs[blk];
    next_there = find.there(e.y, tile, find.v_tok);
  };
  auto place = [&](int buf) {
#pragma unroll
    for (int k = 0; k < KN; ++k) {
      const int u = wave + k * NW;
      if (KU % NW != 0 && u >= KU) break;
      if (W16) {
        kf[buf][2 * u][lane] = centred(kr[k][0], kr[k][1]);
        kf[buf][2 * u + 1][lane] = centred(kr[k][2], kr[k][3]);
      } else {
        kf[buf][u][lane] = centred(kr[k][0], kr[k][1]);
      }
    }
#pragma unroll
    for (int k = 0; k < VN; ++k) {
      const int dt = wave + k * NW;
      if (DT % NW != 0 && dt >= DT) break;
      vf[buf][2 * dt][lane] = centred(vr[k][0], vr[k][1]);
      vf[buf][2 * dt + 1][lane] = centred(vr[k][2], vr[k][3]);
    }
    ks = next_ks;
    sv = next_sv;
    there = next_there;
  };
  if (s0 < s1) {
    entry = find.entries(s0);
    fetch(s0);
    place(0);
    if (s0 + 1 < s1) fetch(s0 + 1);
  }
  int buf = 0;
  for (int tile = s0; tile < s1; ++tile, buf ^= 1) {
    __syncthreads();   // this tile's fragments are there, and the other buffer's readers are done
    const Steps st(ks, sv, there);
    if (tile + 1 < s1) {
      place(buf ^ 1);
      if (tile + 2 < s1) fetch(tile + 2);
    }
    if (tile * kTile >= w_hi || tile * kTile + kTile <= w_lo) continue;
    const int tok = tile * kTile + 16 * g;
    f32x4 s[QT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) s[qt][i] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < DB; ++k) {
        const half8 k8 = kf[buf][i * DB + k][lane];
#pragma unroll
        for (int qt = 0; qt < QT; ++qt)
          s[qt][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k8, w[qt].q[k], s[qt][i], 0, 0, 0);
      }
    }
    if constexpr (DB > 2) reads_ahead<4 * DB, QT>();
    half8 p[QT][2];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) probabilities<DB>(w[qt], s[qt], p[qt], st, tok);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const half8 v0 = vf[buf][2 * dt][lane], v1 = vf[buf][2 * dt + 1][lane];
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) w[qt].o[dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p[qt][0], w[qt].o[dt], 0, 0, 0);
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) w[qt].o[dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p[qt][1], w[qt].o[dt], 0, 0, 0);
    }
    if constexpr (DB > 2) reads_ahead<2 * DT, QT>();
  }

#pragma unroll
  for (int qt = 0; qt < QT; ++qt) {
    const float l = xor_sum(w[qt].l);
    const int rr = mine + 16 * qt + col;
    if (rr >= rows) continue;
    const int64_t out = (row0 + rr / G) * a.Hq + h * G + rr % G, part = split * c.T * a.Hq + out;
    const float by = l == 0.0f ? 0.0f : 1.0f / l;
    if (g == 0) {
      if (!alone) sp.rl[part] = make_float2(w[qt].r, l);
      else if (a.lse) a.lse[out] = l == 0.0f ? -INFINITY : (w[qt].r + __builtin_amdgcn_logf(l)) * kLn2;
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const int d = 16 * dt + 4 * g;
      if (d >= c.D) continue;
      if (alone) {
        struct { S v[4]; } y;
#pragma unroll
        for (int j = 0; j < 4; ++j) y.v[j] = from_f32<S>(w[qt].o[dt][j] * by);
        *(u32x2*)((S*)a.out + out * c.D + d) = __builtin_bit_cast(u32x2, y);
      } else {
        *(f32x4*)(sp.o + part * c.D + d) = w[qt].o[dt];
      }
    }
  }
}

// Joins the splits of a row and head that had more than one: a workgroup each, its
// threads in groups of D / 4 that share the splits, so that the loads of many
// splits are in flight at once.  Four waves for one sequence's many splits, one wave for
// many sequences, most of which have few or one.
template <class T>
__global__ __launch_bounds__(256) void join_kernel(AttArgs a, Split sp, int rows_per_tile) {
  typedef typename T::storage S;
  __shared__ __attribute__((aligned(16))) float so[256 * 4];
  __shared__ float sl[128], stop[4];
  const KvArgs& c = a.c;
  const int tid = threadIdx.x;
  uint32_t e = a.first_block + blockIdx.x;   // (b, i, hq)
  const int hq = (int)(e % (uint32_t)a.Hq);
  e /= (uint32_t)a.Hq;
  const int i = (int)(e % (uint32_t)a.max_new);
  const int b = (int)(e / (uint32_t)a.max_new);
  int64_t row0;
  int n;
  rows_of(c, b, row0, n);
  if (i >= n) return;   // and below max_new by the grid
  if (sp.chosen) sp.tiles = *sp.chosen;
  const int G = a.Hq / c.Hkv, len = a.lens[b], rows = taken(a, n) * G;
  const int base = (i * G + hq % G) / rows_per_tile * rows_per_tile;
  int lo, hi, unused;
  seen_by(a, len, n, base / G, lo, unused);
  seen_by(a, len, n, (base + rows_per_tile < rows ? base + rows_per_tile - 1 : rows - 1) / G, unused, hi);
  const int t0 = lo / kTile, nt = hi > lo ? (hi + kTile - 1) / kTile - t0 : 0;
  if (nt <= sp.tiles) return;
  const int active = (nt + sp.tiles - 1) / sp.tiles;
  const int64_t out = (row0 + i) * a.Hq + hq, step = c.T * a.Hq;
  float top = -INFINITY;
  for (int s = tid; s < active; s += blockDim.x) top = fmaxf(top, sp.rl[s * step + out].x);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
  if (blockDim.x > 64) {
    if ((tid & 63) == 0) stop[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(stop[0], stop[1]), fmaxf(stop[2], stop[3]));
  }
  const int quads = c.D / 4, groups = blockDim.x / quads, group = tid / quads, d = 4 * (tid % quads);
  float l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  if (group < groups) {
#pragma unroll 4
    for (int s = group; s < active; s += groups) {
      const float2 x = sp.rl[s * step + out];
      const float by = x.x == top ? 1.0f : __builtin_amdgcn_exp2f(x.x - top);
      l += x.y * by;
      o += *(const f32x4*)(sp.o + (s * step + out) * c.D + d) * by;
    }
    *(f32x4*)&so[group * c.D + d] = o;
    if (d == 0) sl[group] = l;
  }
  __syncthreads();
  if (group != 0) return;
  o = f32x4{0, 0, 0, 0};
  l = 0.0f;
  for (int g = 0; g < groups; ++g) {
    o += *(const f32x4*)&so[g * c.D + d];
    l += sl[g];
  }
  const float by = l == 0.0f ? 0.0f : 1.0f / l;
  struct { S v[4]; } y;
#pragma unroll
  for (int j = 0; j < 4; ++j) y.v[j] = from_f32<S>(o[j] * by);
  *(u32x2*)((S*)a.out + out * c.D + d) = __builtin_bit_cast(u32x2, y);
  if (d == 0 && a.lse) a.lse[out] = l == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(l)) * kLn2;
}

// How a call is split, from its sizes alone.
struct Plan {
  bool shared;       // attention_rows_kernel
  bool chosen;       // the kernel chooses the tiles of a split
  int64_t blocks;
  int slots;         // workgroups that run at once on 256 compute units
  int QT, NW, splits, tiles, row_tiles, tile_rows;
};

Plan plan(int64_t B, int Hq, int Hkv, int D, int max_new, int max_len) {
  Plan p;
  const int64_t rows = (int64_t)max_new * (Hq / Hkv);
  const int tiles = (max_len + kTile - 1) / kTile;
  p.shared = rows > 64;
  p.QT = rows > 16 && D <= 192 ? 2 : 1;    // wider heads' two row tiles do not fit the registers
  p.NW = 4;
  p.tile_rows = p.shared ? 32 * p.NW : 16 * p.QT;
  p.row_tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
  const int64_t groups = B * Hkv * (int64_t)p.row_tiles;
  const int wide = (D + 31) / 32;
  // Two workgroups on a compute unit, one where the registers or LDS hold no more (256 columns,
  // 8 sequences: 36 us with 256 against 60 with 512; counting the four that 64 columns
  // would allow splits too finely, 21.6 against 19.0 us).
  p.slots = 256 * (wide <= (p.shared || p.QT == 2 ? 4 : 6) ? 2 : 1);
  // Few short sequences: eight waves a workgroup and no second launch.
  // not for heads wider than 192, whose registers eight waves have no room for (513 tokens, 32
  // heads of 256 columns: 24 us with eight, 15 with four; 8 x 1000 tokens, 8 heads: 34 and 19)
  if (p.QT == 1 && groups <= 256 && tiles <= 16 && D <= 192) p.NW = 8;
  p.chosen = B > 1 && B <= 64 * p.NW && !p.shared && p.NW == 4 && tiles > 8;
  if (p.chosen) {
    // lengths differ: the kernel chooses among kChoices powers of two, up to what all
    // sequences at their longest would take
    p.tiles = 8;
    while (p.tiles << (kChoices - 1) < 2 * tiles * groups / p.slots && p.tiles < tiles) p.tiles *= 2;
    while (tiles / p.tiles * groups > 8192) p.tiles *= 2;     // bounds the workspace
    p.blocks = p.slots + groups;   // splits that run at once, or half of that and one for each sequence
  } else if (B > 64 * p.NW && !p.shared) {
    // enough sequences to fill the chip: splits only bound what the longest take (16 tiles a
    // wave, about 35 us), eight of them at most (the workspace)
    p.tiles = tiles > 512 ? (tiles + 31) / 32 * 4 : 64;
  } else {
    // as many workgroups as run at once
    int64_t want = groups >= p.slots ? 1 : p.slots / groups;
    const int per = p.shared ? 1 : p.NW;   // tiles are dealt to a workgroup's waves, or shared by them
    const int64_t most = (tiles + 2 * p.NW - 1) / (2 * p.NW);
    want = want < most ? want : most;
    p.tiles = (int)((tiles + want - 1) / want);
    p.tiles = (p.tiles + per - 1) / per * per;
  }
  p.splits = (tiles + p.tiles - 1) / p.tiles;
  p.chosen = p.chosen && p.splits > 1;
  if (!p.chosen) p.blocks = groups * p.splits;
  return p;
}

template <class T, int DB, int QT, int NW>
void go_w(const AttArgs& a, const Split& sp, unsigned grid, hipStream_t st) {
  if constexpr (DB % 2 == 0) {
    if (a.c.D % 64 == 0) {
      attention_kernel<T, DB, QT, NW, true><<<grid, NW * 64, 0, st>>>(a, sp);
      return;
    }
  }
  attention_kernel<T, DB, QT, NW, false><<<grid, NW * 64, 0, st>>>(a, sp);
}

template <class T, int DB>
void go_q(const AttArgs& a, const Plan& p, const Split& sp, unsigned grid, hipStream_t st) {
  if (p.shared) {
    if constexpr (DB % 2 == 0) {
      if (a.c.D % 64 == 0) {
        attention_rows_kernel<T, DB, 4, true><<<grid, 256, 0, st>>>(a, sp);
        return;
      }
    }
    attention_rows_kernel<T, DB, 4, false><<<grid, 256, 0, st>>>(a, sp);
    return;
  }
  if constexpr (DB <= 6) {
    if (p.QT == 2) return go_w<T, DB, 2, 4>(a, sp, grid, st);
    if (p.NW == 8) return go_w<T, DB, 1, 8>(a, sp, grid, st);
  }
  go_w<T, DB, 1, 4>(a, sp, grid, st);
}

template <class T>
hipError_t go(AttArgs a, const Plan& p, const Split& sp, hipStream_t st) {
  ProfScope prof("awq_kv_attention", st);
  in_parts(p.blocks, 64 * p.NW, [&](uint32_t first, unsigned grid) {
    a.first_block = first;
    switch ((a.c.D + 31) / 32) {
      case 1: go_q<T, 1>(a, p, sp, grid, st); break;
      case 2: go_q<T, 2>(a, p, sp, grid, st); break;
      case 3: go_q<T, 3>(a, p, sp, grid, st); break;
      case 4: go_q<T, 4>(a, p, sp, grid, st); break;
      case 5: go_q<T, 5>(a, p, sp, grid, st); break;
      case 6: go_q<T, 6>(a, p, sp, grid, st); break;
      case 7: go_q<T, 7>(a, p, sp, grid, st); break;
      default: go_q<T, 8>(a, p, sp, grid, st); break;
    }
  });
  return hipGetLastError();
}

template <class T>
hipError_t go_join(AttArgs a, const Plan& p, const Split& sp, hipStream_t st) {
  ProfScope prof("awq_kv_attention_join", st);
  const int threads = p.chosen ? 64 : 256;
  in_parts((int64_t)a.c.B * a.max_new * a.Hq, threads, [&](uint32_t first, unsigned grid) {
    a.first_block = first;
    join_kernel<T><<<grid, threads, 0, st>>>(a, sp, p.tile_rows);
  });
  return hipGetLastError();
}

}  // namespace

size_t kv_attention_ws_bytes(int64_t T, int64_t B, int Hq, int Hkv, int D, int max_new,
                             int max_len) {
  const Plan p = plan(B, Hq, Hkv, D, max_new, max_len);
  return p.splits == 1 ? 0 : (size_t)p.splits * T * Hq * (D + 2) * 4 + 4;
}

// Covers every call of these heads with at most these T, B, max_new and max_len whose rows
// are at most its own B max_new, and this one whatever its page table holds.  In rows of
// partial results, splits times rows of a call are, by plan():
//   any: a split takes at least eight tiles, so at most `most` times its rows;
//   as many workgroups as run at once: splits times groups are at most 512, and rows at most
//     groups times a row tile;
//   chosen by the kernel (up to 64 rows a group, 2 to 256 sequences): whole splits times groups
//     at most 8192, and one more;
//   more sequences: at most eight splits.
size_t kv_attention_ws_bound(int64_t T, int64_t B, int Hq, int Hkv, int D, int max_new,
                             int max_len) {
  const int64_t most = ((max_len + kTile - 1) / kTile + 7) / 8, G = Hq / Hkv;
  if (most <= 1) return 0;
  const auto upto = [&](int64_t rows, int64_t cap) { return rows > cap / most ? cap : rows * most; };
  const int64_t tile = D <= 192 ? 32 : 16;
  int64_t n = upto(T * Hq, 512 * (max_new * G > 64 ? 128 : tile));
  if (G <= 64) {
    const int64_t few = 64 / G;     // rows of a sequence that make 64 of a group
    if (B > 1) {
      const int64_t rows = std::min(T, std::min<int64_t>(B, 256) * few) * Hq;
      n = std::max(n, upto(rows, 8192 * tile + rows));
    }
    if (B > 256) n = std::max(n, std::min(T, B * few) * Hq * std::min<int64_t>(most, 8));
  }
  if (T > B * max_new) {            // rows that no sequence may have are counted all the same
    const int64_t groups = B * Hkv * plan(B, Hq, Hkv, D, max_new, max_len).row_tiles;
    n = std::max(n, std::min(most, 8192 / groups + 9) * T * Hq);
  }
  return (size_t)n * (D + 2) * 4 + 4;
}

int64_t kv_attention_blocks(int64_t B, int Hq, int Hkv, int D, int max_new, int max_len) {
  if (max_new > (int64_t)INT32_MAX / Hq) return INT64_MAX;
  const Plan p = plan(B, Hq, Hkv, D, max_new, max_len);
  return p.splits == 1 ? p.blocks : std::max(p.blocks, B * max_new * Hq);
}

hipError_t launch_kv_attention(const AttArgs& a, awq_dtype_t dt, void* ws, hipStream_t st) {
  const Plan p = plan(a.c.B, a.Hq, a.c.Hkv, a.c.D, a.max_new, a.max_len);
  Split sp = {p.splits, p.tiles, p.row_tiles, p.slots, nullptr, nullptr, nullptr};
  if (p.splits > 1) {
    sp.o = (float*)ws;
    sp.rl = (float2*)(sp.o + (size_t)p.splits * a.c.T * a.Hq * a.c.D);
    if (p.chosen) sp.chosen = (int*)(sp.rl + (size_t)p.splits * a.c.T * a.Hq);
  }
  const hipError_t e = dt == AWQ_F16 ? go<F16T>(a, p, sp, st) : go<BF16T>(a, p, sp, st);
  if (e != hipSuccess || p.splits == 1) return e;
  return dt == AWQ_F16 ? go_join<F16T>(a, p, sp, st) : go_join<BF16T>(a, p, sp, st);
}

}  // namespace awq
