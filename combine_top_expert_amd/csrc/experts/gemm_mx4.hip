// moe_grouped_gemm_mx4: the experts' products of MX4 rows and MX4 weights.
//
// G[q,n] = sum over blocks b of 32 columns of 2^(sa[q,b] + sw[n,b] - 254) sum_{k in b} A[q,k] W[n,k].
// The matrix cores take both operands' 4-bit codes and scale bytes as they are
// (16 x 16 x 128, a scale per 32) and add to fp32 sums, so a product has no
// conversion and no fold.
//
// Tiles of up to 256 rows x 256 columns, one workgroup of 8 waves per CU.
//  - Weights go from memory straight into registers: a wave owns 32 columns of
//    the tile, so no other wave of the workgroup needs them, and they are packed
//    in the order of the operand's registers (1 KB a load).
//  - Rows are shared by the 8 waves and go through LDS, 256 columns a stage,
//    three stages in turn with one barrier each; their scales are turned so that
//    a lane reads those of four 128-column steps as one dword, a byte of which
//    the instruction picks.
//  - Weights are the first operand: a lane's four sums are then four
//    neighbouring columns of one row.
//  - With SiLU a wave owns 16 gate columns and their 16 up columns, so the
//    product forms in registers; a block of 32 columns of MX4 output belongs to two
//    neighbouring waves, which exchange their maxima through LDS.
// An expert's rows are cut into row blocks of nearly equal size, a multiple of
// 16, and a tile's loop is built for the number of 16-row groups it has (1, 2, 4,
// .. 16): the shorter its stages, the more of them are loaded ahead.
//
// Bound by the loads that a CU's memory path holds at a time, about 100 of 128
// bytes (counters at 4 / 128 rows an expert: 104 / 85 in flight, 1315 / 770 cycles
// each): with few rows that is the weights' stream, at 6.2 to 6.6 TB/s in gate/up and 5.1
// in the shorter down product; with more, the reads of rows and of their scales from L2
// take places in it.  The scales take as many as the rows do, a quarter of all at 128
// rows, as each thread opens a line of its own for 16 bytes.  At 512 rows the matrix cores
// come to 56 % of what they reach on random codes (6.5 PFLOP/s; 8.5 on constant ones).
// Measured, us, 32 experts with the same number of rows, 4 / 16 / 32 / 64 / 128 / 256 / 512:
// gate/up 4096 x 7168 (500 MB) 77 / 79 / 81 / 90 / 109 / 153 / 268 (3.6 PFLOP/s); down 7168 x
// 2048 (250 MB) 49 / 51 / 54 / 60 / 75 / 111 / 190.  One decode step (128 tokens, about 70 rows,
// 28 experts) 69 and 45.
// What else was measured: weights through the caches 78 at decode (68 non-temporal);
// weight scales shifted where they are loaded, 20 us more at 4 rows (a wait of a memory
// round trip every four steps); row loads behind a branch at K's end, 2 to 8 % more;
// one stream of loads over all tiles of a workgroup, the last tiles cut into column
// parts, and more stages of weights ahead (4 at 10 and 12 groups, 8 at 1 and 2): no gain.

#include <type_traits>

#include "experts_common.h"

namespace {

using namespace moe_experts;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * MOE_WAVE;
constexpr int kRows = 256;                         // most rows of a tile
constexpr int kCols = kWaves * 32;                 // weight rows (G columns) of a tile
constexpr int kGrid = 256;                         // workgroups: one a CU
constexpr int kBand = 8;                           // row blocks that share a pass over an expert's columns
constexpr int kMaxExperts = 1024;

enum Epilogue { kStoreF32, kStoreBf16, kSiluF32, kSiluBf16, kSiluMx4 };
constexpr bool is_silu(int e) { return e >= kSiluF32; }

struct GemmArgs {
  const uint8_t* a;
  const uint8_t* as;
  const uint8_t* w;
  const uint8_t* ws;
  const int32_t* counts;
  const int32_t* offsets;
  int L;
  int64_t rows_cap;
  int N, K;
  void* out;
  uint8_t* out_scales;
};

struct Tile {
  int expert, col, rows;                           // col: first of the tile's 16-column groups (of gate columns with SiLU)
  int64_t row;                                     // first row in the buffer
};

struct Shared {
  u32x4 a[3][kRows * 8];                           // [row][8 chunks of 16 bytes, swizzled]
  uint32_t as[2][kRows * 4];                       // [row][32-column block of a step] x 4 steps
  float top[kWaves][kRows];
  int begin[kMaxExperts + 1];                      // row blocks before expert e
  int rows[kMaxExperts], first[kMaxExperts];       // its valid rows, and where they begin
  int part[kWaves];
};

__device__ __forceinline__ i32x8 operand(const u32x4& v) {
  return i32x8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]), static_cast<int>(v[3]), 0, 0, 0, 0};
}
template <int S> __device__ __forceinline__ f32x4 mma(const u32x4& w, const u32x4& a, const f32x4& c, uint32_t sw, uint32_t sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(a), c, 4, 4, S, static_cast<int>(sw), S,
                                                          static_cast<int>(sa));
}
// The place of chunk c of row r.  The two chunks that lane group g reads of a row, g and 4 + g, are
// neighbours, and swizzled so that the 16 lanes which a 16-byte LDS read serves at a time (they are of
// two lane groups) meet no bank twice.
__device__ __forceinline__ int place(int r, int c) { return r * 8 + (((c & 3) << 1 | c >> 2) ^ (r & 7) ^ (r >> 3 & 1)); }

// valid rows of expert e, in the buffer
__device__ __forceinline__ int rows_of(const GemmArgs& p, int e) {
  const int64_t at = p.offsets[e];
  int64_t n = p.counts[e];
  if (at < 0 || at >= p.rows_cap) return 0;
  n = n < p.rows_cap - at ? n : p.rows_cap - at;
  return static_cast<int>(n > 0 ? n : 0);
}

// v as if it were not known: what follows from it is worked out where it is used, rather than kept in
// registers over the tiles
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// sh.begin[e] = row blocks, of at most `limit` rows, of the experts before e; all of them are returned.  The
// first call (FIRST) also fills sh.rows and sh.first.
template <bool FIRST> __device__ __forceinline__ int count_blocks(const GemmArgs& p, Shared& sh, int limit) {
  const int lane = moe::lane_id(), wave = threadIdx.x >> 6;
  int base = 0;
  for (int e0 = 0; e0 < p.L; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    const int rows = e < p.L ? (FIRST ? rows_of(p, e) : sh.rows[e]) : 0, mine = (rows + limit - 1) / limit;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(sum, d);
      if (lane >= d) sum += o;
    }
    if (lane == 63) sh.part[wave] = sum;
    __syncthreads();
    int before = base;
    for (int w = 0; w < kWaves; ++w) {
      const int v = sh.part[w];
      if (w < wave) before += v;
      base += v;
    }
    if (e < p.L) {
      sh.begin[e] = before + sum - mine;
      if constexpr (FIRST) sh.rows[e] = rows, sh.first[e] = p.offsets[e];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) sh.begin[p.L] = base;
  __syncthreads();
  return uniform(base);
}

// A workgroup's tiles: every 32nd from `at` on.  Of `groups` 16-column groups of a tile (of gate
// columns with SiLU) it takes one of 2^split parts, which the first 8 >> split waves have.
struct Walk {
  int64_t at, end;
  int ncol, groups, split, wave;
};

// the most rows that an expert has
__device__ __forceinline__ int most_rows(const GemmArgs& p, Shared& sh) {
  int m = 0;
  for (int e = threadIdx.x; e < p.L; e += kThreads) m = max(m, sh.rows[e]);
#pragma unroll
  for (int d = 32; d > 0; d /= 2) m = max(m, __shfl_xor(m, d));
  if (moe::lane_id() == 0) sh.part[threadIdx.x >> 6] = m;
  __syncthreads();
  for (int w = 0; w < kWaves; ++w) m = max(m, sh.part[w]);
  __syncthreads();
  return uniform(m);
}

__device__ __forceinline__ Tile tile_at(const GemmArgs& p, const Shared& sh, const Walk& w) {
  const int ncol = w.ncol;
  const int64_t t = w.at >> w.split;
  int lo = 0, hi = p.L - 1;                        // the last expert whose tiles begin at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(uniform(sh.begin[mid])) * ncol <= t) lo = mid;
    else hi = mid - 1;
  }
  const int begin = uniform(sh.begin[lo]), blocks = uniform(sh.begin[lo + 1]) - begin, rows = uniform(sh.rows[lo]);
  int64_t r = t - static_cast<int64_t>(begin) * ncol;
  const int band = blocks > kBand ? static_cast<int>(r / (static_cast<int64_t>(kBand) * ncol)) : 0;
  r -= static_cast<int64_t>(band) * kBand * ncol;  // below kBand * ncol
  const uint32_t high = blocks - band * kBand < kBand ? blocks - band * kBand : kBand;
  const uint32_t col = static_cast<uint32_t>(r) / high;
  const int block = band * kBand + static_cast<int>(static_cast<uint32_t>(r) - col * high);
  const int each = (static_cast<int>(static_cast<uint32_t>(rows + blocks - 1) / static_cast<uint32_t>(blocks)) + 15) & ~15;
  const int first = block * each;
  const int part = static_cast<int>(w.at) & ((1 << w.split) - 1);
  return Tile{lo, static_cast<int>(col) * w.groups + part * (w.groups >> w.split), rows - first < each ? rows - first : each,
              static_cast<int64_t>(uniform(sh.first[lo])) + first};
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return static_cast<uint32_t>(moe::f32_to_bf16(a)) | static_cast<uint32_t>(moe::f32_to_bf16(b)) << 16;
}
// four neighbouring columns of a row
__device__ __forceinline__ void store4(float* out, const f32x4& v) {
  *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(uint16_t* out, const f32x4& v) {
  const uint2 d = make_uint2(
      static_cast<uint32_t>(moe::f32_to_bf16(v[0])) | static_cast<uint32_t>(moe::f32_to_bf16(v[1])) << 16,
      static_cast<uint32_t>(moe::f32_to_bf16(v[2])) | static_cast<uint32_t>(moe::f32_to_bf16(v[3])) << 16);
  *reinterpret_cast<uint2*>(out) = d;
}

typedef __amdgpu_buffer_rsrc_t rsrc_t;
// num: the bytes from base on that may be read; what lies behind them reads as 0
__device__ __forceinline__ rsrc_t resource(const uint8_t* base, uint32_t num) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, static_cast<int>(num), 0x00020000);
}

// Where a wave reads a tile's operands, and what it has loaded of them before the tile begins
struct Operands {
  rsrc_t rows, scales;                             // of the tile's valid rows only
  rsrc_t w[2];                                     // this wave's two groups of 16 weight rows
  const uint8_t* ws[2];
  int last[2];                                     // bytes of scales in the buffer from the group's first on, less 4
  bool live;                                       // the wave has columns in this tile
};
struct Loaded {
  u32x4 rows[2][4];                                // of two stages
  u32x4 scales;                                    // of four steps
  u32x4 w[2][2][2];                                // [stage][step][group]
  uint32_t ws[2];
};

template <int EPI> __device__ __forceinline__ Operands operands(const GemmArgs& p, const Tile& t, const Walk& w) {
  const int wave = w.wave;
  const int steps = p.K >> 7, tiles = p.N >> 4, half = tiles >> 1;
  const int n0 = is_silu(EPI) ? t.col + wave : t.col + 2 * wave;
  const int n1 = is_silu(EPI) ? n0 + half : n0 + 1;
  Operands o;
  o.live = wave < kWaves >> w.split && n1 < tiles && (!is_silu(EPI) || n0 < half);
  o.rows = resource(p.a + t.row * (p.K >> 1), static_cast<uint32_t>(t.rows) * static_cast<uint32_t>(p.K >> 1));
  o.scales = resource(p.as + t.row * (p.K >> 5), static_cast<uint32_t>(t.rows) * static_cast<uint32_t>(p.K >> 5));
  const int64_t all = static_cast<int64_t>(p.L) * tiles;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t g = static_cast<int64_t>(t.expert) * tiles + (o.live ? (j ? n1 : n0) : 0);
    o.w[j] = resource(p.w + g * steps * 1024, o.live ? static_cast<uint32_t>(steps) * 1024u : 0u);
    o.ws[j] = p.ws + g * steps * 64;
    o.last[j] = g < all - 1 ? 0x7fffffff : steps * 64 - 4;
  }
  return o;
}

// Codes of a step; zeros behind K's end, where nothing is read.  Non-temporal (2): a decode step reads each
// once, and with few row blocks they are read at about the same time (gate/up decode 78 -> 68 us, prefill
// 125 -> 118).
__device__ __forceinline__ u32x4 load_weight(const Operands& o, int lane, int step, int j) {
  return __builtin_amdgcn_raw_buffer_load_b128(o.w[j], lane * 16, step * 1024, 2);
}
__device__ __forceinline__ void load_weights(const Operands& o, int lane, int stage, u32x4 (&r)[2][2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 2; ++j) r[h][j] = load_weight(o, lane, stage * 2 + h, j);
}

// The scales of four steps.  The places of the last, shorter group are not dwords: what is read behind
// them is masked later, and at the buffer's end the dword begins earlier.
__device__ __forceinline__ void load_weight_scales(const Operands& o, int quad, int steps, uint32_t (&d)[2]) {
  const int there = quad * 4 < steps ? quad : (steps - 1) >> 2;      // behind the last: that one again
  const int n = steps - there * 4 < 4 ? steps - there * 4 : 4, off = there * 256 + moe::lane_id() * n;
#pragma unroll
  for (int j = 0; j < 2; ++j) __builtin_memcpy(&d[j], o.ws[j] + (off < o.last[j] ? off : o.last[j]), 4);
}
// as loaded -> byte s for step s, 0 for steps that do not exist
__device__ __forceinline__ uint32_t weight_scales(const Operands& o, int quad, int steps, uint32_t d, int j) {
  const int left = steps - quad * 4, n = left < 0 ? 0 : left < 4 ? left : 4, off = quad * 256 + moe::lane_id() * n;
  const uint32_t mask = n == 4 ? ~0u : (1u << (8 * n)) - 1;
  return d >> (8 * (off < o.last[j] ? 0 : off - o.last[j]) & 31) & mask;
}

// This thread's part of a stage's rows: chunk tid & 7 of row (tid >> 3) + 64 i.  Rows behind the tile's last and
// stages behind K's end read as 0 or as other columns (whose scales are 0), without a branch: branches
// among the products cost registers.
__device__ __forceinline__ u32x4 load_row(const GemmArgs& p, const Operands& o, int tid, int stage, int i) {
  const uint32_t half = static_cast<uint32_t>(p.K >> 1);
  const uint32_t at = stage * 256 < p.K ? 64 * i * half + stage * 128 : 0x7fff0000u;
  return __builtin_amdgcn_raw_buffer_load_b128(o.rows, static_cast<int>((tid >> 3) * half + (tid & 7) * 16),
                                               static_cast<int>(at), 0);
}
// and of four steps' scales: those of row tid, modulo the tile's (two threads carry the same)
__device__ __forceinline__ u32x4 load_scales(const GemmArgs& p, const Operands& o, int tid, int quad) {
  return __builtin_amdgcn_raw_buffer_load_b128(o.scales, static_cast<int>((tid & (kRows - 1)) * static_cast<uint32_t>(p.K >> 5)),
                                               quad * 16, 0);
}

// What a tile needs first; issued before the epilogue of the tile before it
__device__ __forceinline__ Loaded load_first(const GemmArgs& p, const Operands& o) {
  const int steps = p.K >> 7;
  Loaded l;
  load_weight_scales(o, 0, steps, l.ws);
  const int tid = fresh(threadIdx.x);
  l.scales = load_scales(p, o, tid, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l.rows[0][i] = load_row(p, o, tid, 0, i);
    l.rows[1][i] = load_row(p, o, tid, 1, i);
  }
  load_weights(o, tid & 63, 0, l.w[0]);
  load_weights(o, tid & 63, 1, l.w[1]);
  return l;
}

// The products of a tile of MB groups of 16 rows.  `l` holds its first loads.
template <int MB>
__device__ __forceinline__ void multiply(const GemmArgs& p, Shared& sh, const Operands& o, const Loaded& l, f32x4 (&acc)[MB][2]) {
  const int tid = fresh(threadIdx.x), lane = tid & 63;
  const int steps = p.K >> 7, stages = (steps + 1) >> 1;
  const int q = lane & 15, g = lane >> 4;
  // How far ahead of their use weights, rows and scales are loaded: more where a stage is short.
  constexpr int kAhead = MB <= 8 ? 4 : 2;          // stages of weights in registers
  constexpr int kRowSets = MB <= 4 ? 4 : MB <= 8 ? 2 : 1;   // stages of rows on their way to LDS
  constexpr int kQuads = MB <= 8 ? 2 : 1;          // quads of scales
  constexpr int kLoads = (MB * 16 + 63) / 64;
  constexpr bool kSpread = MB >= 8;                // loads between products, not in one run

  u32x4* const store_at = &sh.a[0][place(tid >> 3, tid & 7)];
  auto store_row = [&](int b, int i, const u32x4& r) { store_at[b * (kRows * 8) + i * 512] = r; };
  // scales of a row: [step][block] bytes to [block][step], zeros behind K's end
  auto store_scales = [&](int quad, u32x4 s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = quad * 4 + j < steps ? s[j] : 0u;
    const uint32_t lo0 = __builtin_amdgcn_perm(s[1], s[0], 0x05010400u), hi0 = __builtin_amdgcn_perm(s[1], s[0], 0x07030602u);
    const uint32_t lo1 = __builtin_amdgcn_perm(s[3], s[2], 0x05010400u), hi1 = __builtin_amdgcn_perm(s[3], s[2], 0x07030602u);
    reinterpret_cast<u32x4*>(sh.as[quad & 1])[tid & (kRows - 1)] = u32x4{
        __builtin_amdgcn_perm(lo1, lo0, 0x05040100u), __builtin_amdgcn_perm(lo1, lo0, 0x07060302u),
        __builtin_amdgcn_perm(hi1, hi0, 0x05040100u), __builtin_amdgcn_perm(hi1, hi0, 0x07060302u)};
  };

  u32x4 wr[kAhead][2][2], ar[kRowSets][kLoads], sr[kQuads];
  uint32_t sw[kQuads][2];
#pragma unroll
  for (int i = 1; i <= kQuads; ++i) sr[i % kQuads] = load_scales(p, o, tid, i);
#pragma unroll
  for (int i = 0; i < kRowSets; ++i)
#pragma unroll
    for (int k = 0; k < kLoads; ++k) ar[i][k] = load_row(p, o, tid, 2 + i, k);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) wr[i][h][0] = l.w[i][h][0], wr[i][h][1] = l.w[i][h][1];
#pragma unroll
  for (int i = 2; i < (kSpread ? kAhead - 1 : kAhead); ++i)
    load_weights(o, lane, i, wr[i]);
  sw[0][0] = l.ws[0], sw[0][1] = l.ws[1];
  if (kQuads > 1) load_weight_scales(o, 1, steps, sw[kQuads - 1]);
#pragma unroll
  for (int k = 0; k < kLoads; ++k) store_row(0, k, l.rows[0][k]), store_row(1, k, l.rows[1][k]);
  store_scales(0, l.scales);
#pragma unroll
  for (int m = 0; m < MB; ++m) acc[m][0] = acc[m][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();

  // Fragments are fetched kFetch row groups before their products, the first ones of a stage during the
  // stage before it.
  constexpr int kFetch = MB > 1 ? 2 : 1;
  struct Frag { u32x4 f0, f1; uint32_t s; };
  const u32x4* frag = &sh.a[0][place(q, g)];       // chunk g of row q; chunk 4 + g is its neighbour, either way
  const int across = place(q, 4 + g) - place(q, g);
  Frag next[kFetch];
  auto fetch = [&](const u32x4* from, const uint32_t* scales, int m) {
    return Frag{from[m * 128], from[m * 128 + across], scales[m * 64]};
  };
  auto scales_at = [&](int stage) { return &sh.as[stage >> 1 & 1][q * 4 + g]; };
#pragma unroll
  for (int i = 0; i < kFetch; ++i) next[i] = fetch(frag, scales_at(0), i);

  // One barrier a stage: when stage s begins, the rows of stage s + 1 are in LDS, those of stage s - 1
  // have been read, and s + 2 takes their place.  Steps behind K's last are multiplied like the others:
  // both their scales are 2^-127, which leaves nothing of any code.
  uint32_t c0 = 0, c1 = 0;
  int b0 = 0, b1 = 1, b2 = 2;                      // the buffers of stages s, s + 1, s + 2
#pragma unroll 1
  for (int first = 0; first < stages; first += kAhead) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int stage = first + j, quad = stage >> 1;
      if (j % 2 == 0) {
        uint32_t (&d)[2] = sw[j / 2 % kQuads];
        c0 = weight_scales(o, quad, steps, d[0], 0), c1 = weight_scales(o, quad, steps, d[1], 1);
        load_weight_scales(o, quad + kQuads, steps, d);
      }
      const u32x4* here = frag + b0 * (kRows * 8);
      const u32x4* there = frag + b1 * (kRows * 8);
      const uint32_t* here_s = scales_at(stage);
      const uint32_t* there_s = scales_at(stage + 1);
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const Frag f = next[0];
        if constexpr (kFetch == 2) next[0] = next[1];
        next[kFetch - 1] = m + kFetch < MB ? fetch(here, here_s, m + kFetch) : fetch(there, there_s, m + kFetch - MB);
        if (j % 2 == 0) {
          acc[m][0] = mma<0>(wr[j][0][0], f.f0, acc[m][0], c0, f.s);
          acc[m][1] = mma<0>(wr[j][0][1], f.f0, acc[m][1], c1, f.s);
          acc[m][0] = mma<1>(wr[j][1][0], f.f1, acc[m][0], c0, f.s);
          acc[m][1] = mma<1>(wr[j][1][1], f.f1, acc[m][1], c1, f.s);
        } else {
          acc[m][0] = mma<2>(wr[j][0][0], f.f0, acc[m][0], c0, f.s);
          acc[m][1] = mma<2>(wr[j][0][1], f.f0, acc[m][1], c1, f.s);
          acc[m][0] = mma<3>(wr[j][1][0], f.f1, acc[m][0], c0, f.s);
          acc[m][1] = mma<3>(wr[j][1][1], f.f1, acc[m][1], c1, f.s);
        }
        // products and fetches stay in this order
        if constexpr (MB > 1)
          asm volatile("" : "+v"(acc[m][0]), "+v"(acc[m][1]), "+v"(acc[(m + 1) % MB][0]), "+v"(acc[(m + 1) % MB][1])::"memory");
        else
          asm volatile("" : "+v"(acc[m][0]), "+v"(acc[m][1])::"memory");
        if constexpr (kSpread) {
          if (m >= 1 && m <= 4) {                  // one of the four weight loads of stage + kAhead - 1
            const int h = (m - 1) >> 1, w = (m - 1) & 1;
            wr[(j + kAhead - 1) % kAhead][h][w] = load_weight(o, lane, (stage + kAhead - 1) * 2 + h, w);
          }
          if (m >= 5 && m % 2 == 1 && (m - 5) / 2 < kLoads) {
            const int i = (m - 5) / 2;
            store_row(b2, i, ar[j % kRowSets][i]);
            ar[j % kRowSets][i] = load_row(p, o, tid, stage + 2 + kRowSets, i);
          }
        }
        if (m == (kSpread ? 6 : 0)) {
          if (!kSpread) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
              store_row(b2, i, ar[j % kRowSets][i]);
              ar[j % kRowSets][i] = load_row(p, o, tid, stage + 2 + kRowSets, i);
            }
          }
          if (j % 2 == 0) {
            store_scales(quad + 1, sr[(j / 2 + 1) % kQuads]);
            sr[(j / 2 + 1) % kQuads] = load_scales(p, o, tid, quad + 1 + kQuads);
          }
        }
      }
      if constexpr (!kSpread) load_weights(o, lane, stage + kAhead, wr[j]);
      const int b = b0;
      b0 = b1, b1 = b2, b2 = b;
      __syncthreads();
    }
  }
}

template <int MB, int EPI>
__device__ __forceinline__ void epilogue(const GemmArgs& p, Shared& sh, const Tile& t, bool live, f32x4 (&acc)[MB][2]) {
  const int lane = fresh(moe::lane_id());
  const int wave = uniform(static_cast<int>(threadIdx.x >> 6)), q = lane & 15, g = lane >> 4;
  const int n0 = is_silu(EPI) ? t.col + wave : t.col + 2 * wave;
  // lane (q, g) holds row m * 16 + q, columns 4 g .. 4 g + 3 of each group
  if constexpr (is_silu(EPI)) {
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][0][i] = moe::silu(acc[m][0][i]) * acc[m][1][i];
  }
  const int cols = is_silu(EPI) ? p.N >> 1 : p.N;
  if constexpr (EPI == kSiluMx4) {
    // a row's 16 columns are in 4 lanes, 16 apart; the other 16 of its block in the neighbouring wave
    uint32_t top[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      uint32_t v = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) v = max(v, magnitude(acc[m][0][i]));
      const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      v = max(r[0], r[1]);
      const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
      top[m] = max(s[0], s[1]);
      if (g == 0) sh.top[wave][m * 16 + q] = __uint_as_float(top[m]);
    }
    __syncthreads();
    if (live) {
      uint32_t code[MB];
      uint8_t* os = p.out_scales + (t.row + q) * (cols >> 5) + (n0 >> 1);
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const int row = m * 16 + q;
        const uint32_t s = mx4_scale(max(top[m], __float_as_uint(sh.top[wave ^ 1][row])));
        const float v[4] = {acc[m][0][0], acc[m][0][1], acc[m][0][2], acc[m][0][3]};
        code[m] = mx4_codes4(v, s);
        if (row < t.rows && g == 0 && (wave & 1) == 0) *os = static_cast<uint8_t>(s);
        os += 16 * (cols >> 5);
      }
      uint8_t* out = static_cast<uint8_t*>(p.out) + n0 * 8;
      // four lanes' 2 bytes of four row groups change places: lane group g stores 8 bytes of row group g
      const int64_t pitch = cols >> 1;
#pragma unroll
      for (int m = 0; m + 4 <= MB; m += 4) {
        uint32_t e[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const auto r = __builtin_amdgcn_permlane16_swap(code[m + 2 * h], code[m + 2 * h + 1], false, false);
          e[h] = r[0] | r[1] << 16;
        }
        const auto r = __builtin_amdgcn_permlane32_swap(e[0], e[1], false, false);
        const int row = (m + g) * 16 + q;
        if (row < t.rows) *reinterpret_cast<uint2*>(out + (t.row + row) * pitch) = make_uint2(r[0], r[1]);
      }
#pragma unroll
      for (int m = MB & ~3; m < MB; ++m) {
        const int row = m * 16 + q;
        if (row < t.rows) *reinterpret_cast<uint16_t*>(out + (t.row + row) * pitch + g * 2) = static_cast<uint16_t>(code[m]);
      }
    }
  } else if (live) {
    if constexpr (EPI == kStoreBf16) {
      // lanes 16 apart change places: even lane groups then hold 8 columns of the first group, odd ones of the second
      uint16_t* out = static_cast<uint16_t*>(p.out) + (t.row + q) * cols + n0 * 16 + (g & 1) * 16 + (g >> 1) * 8;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16(acc[m][0][0], acc[m][0][1]), pack_bf16(acc[m][1][0], acc[m][1][1]), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16(acc[m][0][2], acc[m][0][3]), pack_bf16(acc[m][1][2], acc[m][1][3]), false, false);
        if (m * 16 + q < t.rows) *reinterpret_cast<uint4*>(out) = make_uint4(lo[0], hi[0], lo[1], hi[1]);
        out += 16 * static_cast<int64_t>(cols);
      }
    } else if constexpr (EPI == kSiluBf16 && MB % 2 == 0) {
      // likewise over two row groups: even lane groups hold 8 columns of a row of the first, odd ones of the second
      uint16_t* out = static_cast<uint16_t*>(p.out) + (t.row + (g & 1) * 16 + q) * cols + n0 * 16 + (g >> 1) * 8;
#pragma unroll
      for (int m = 0; m < MB; m += 2) {
        const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16(acc[m][0][0], acc[m][0][1]), pack_bf16(acc[m + 1][0][0], acc[m + 1][0][1]), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16(acc[m][0][2], acc[m][0][3]), pack_bf16(acc[m + 1][0][2], acc[m + 1][0][3]), false, false);
        if ((m + (g & 1)) * 16 + q < t.rows) *reinterpret_cast<uint4*>(out) = make_uint4(lo[0], hi[0], lo[1], hi[1]);
        out += 32 * static_cast<int64_t>(cols);
      }
    } else {
      typedef typename std::conditional<EPI == kStoreF32 || EPI == kSiluF32, float, uint16_t>::type T;
      T* out = static_cast<T*>(p.out) + (t.row + q) * cols + n0 * 16 + g * 4;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if (m * 16 + q < t.rows) {
          store4(out, acc[m][0]);
          if constexpr (!is_silu(EPI)) store4(out + 16, acc[m][1]);
        }
        out += 16 * static_cast<int64_t>(cols);
      }
    }
  }
}

// The number of 16-row groups that a tile's loop is built for
__device__ __forceinline__ int groups_of(const Tile& t) {
  const int mb = (t.rows + 15) >> 4;
  return mb <= 2 ? mb : (mb + 1) & ~1;
}

// Tiles of MB row groups, while they follow each other: the products of one, then the first loads of the
// next, then the epilogue of the first.  (What was loaded ahead stays in one loop's registers: carried
// from one variant's loop to another's it would be spilled.)  Returns with w.at at the tile t that is
// another variant's, or behind the end.
template <int MB, int EPI>
__device__ __forceinline__ void run_tiles(const GemmArgs& p, Shared& sh, Walk& w, Tile& t) {
  Operands o = operands<EPI>(p, t, w);
  Loaded l = load_first(p, o);
  for (bool same = true; same;) {
    f32x4 acc[MB][2];
    multiply<MB>(p, sh, o, l, acc);
    const Tile here = t;
    const bool live = o.live;
    w.at += kGrid >> 3;
    same = false;
    if (w.at < w.end) {
      t = tile_at(p, sh, w);
      same = groups_of(t) == MB;
    }
    if (same) {
      o = operands<EPI>(p, t, w);
      l = load_first(p, o);
    } else {
      l = Loaded{};
    }
    epilogue<MB, EPI>(p, sh, here, live, acc);
  }
}

template <int EPI>
__global__ __launch_bounds__(kThreads, 2) void gemm_mx4_kernel(const GemmArgs p) {
  __shared__ Shared sh;
  Walk w;
  w.wave = uniform(static_cast<int>(threadIdx.x >> 6));
  w.groups = is_silu(EPI) ? kWaves : 2 * kWaves;
  w.ncol = ((is_silu(EPI) ? p.N >> 5 : p.N >> 4) + w.groups - 1) / w.groups;
  w.split = 0;
  int64_t tiles = static_cast<int64_t>(count_blocks<true>(p, sh, kRows)) * w.ncol;
  // Too few tiles for the CUs: the longer side of a tile is halved while its parts find a CU each.  (A block of MX4
  // output's two waves stay together.)  Whole tiles against parts, us: 2 experts x about 200 rows, 6272 x 6400, 47 and 34;
  // 2 x 1 row, 2304 x 5632, 19.5 and 18; 16 x about 200 rows, 1152 x 3456, 37 and 34.
  if (tiles > 0 && tiles <= kGrid / 2) {
    const int most = most_rows(p, sh);
    int limit = kRows;
    while (limit > 16 && limit / 2 >= most) limit /= 2;          // the same row blocks
    for (;;) {
      const bool wide = w.split < (EPI == kSiluMx4 ? 2 : 3) && kCols >> w.split >= (most < limit ? most : limit);
      if (wide) {
        if (tiles * 2 > kGrid) break;
        ++w.split, tiles *= 2;
      } else {
        if (limit <= 16) break;
        const int64_t more = static_cast<int64_t>(count_blocks<false>(p, sh, limit / 2)) * w.ncol << w.split;
        if (more > kGrid) {
          count_blocks<false>(p, sh, limit);
          break;
        }
        limit /= 2, tiles = more;
      }
    }
  }
  // workgroup i runs on XCD i mod 8: each XCD takes a contiguous eighth of the
  // tiles, 32 neighbouring ones at a time, which share rows and weights in its L2
  const int64_t per = (tiles + 7) >> 3, lo = (blockIdx.x & 7) * per;
  w.end = lo + per < tiles ? lo + per : tiles;
  w.at = lo + (blockIdx.x >> 3);
  if (w.at >= w.end) return;
  Tile t = tile_at(p, sh, w);
  while (w.at < w.end) {
    switch (groups_of(t)) {
      case 1: run_tiles<1, EPI>(p, sh, w, t); break;
      case 2: run_tiles<2, EPI>(p, sh, w, t); break;
      case 4: run_tiles<4, EPI>(p, sh, w, t); break;
      case 6: run_tiles<6, EPI>(p, sh, w, t); break;
      case 8: run_tiles<8, EPI>(p, sh, w, t); break;
      case 10: run_tiles<10, EPI>(p, sh, w, t); break;
      case 12: run_tiles<12, EPI>(p, sh, w, t); break;
      case 14: run_tiles<14, EPI>(p, sh, w, t); break;
      default: run_tiles<16, EPI>(p, sh, w, t); break;
    }
  }
}

}  // namespace

extern "C" moe_status moe_grouped_gemm_mx4(const void* a, const void* a_scales, const void* codes_packed,
                                           const void* scales_packed, const int32_t* counts, const int32_t* offsets,
                                           int L, int64_t rows_cap, int N, int K, moe_w13_epilogue epi, void* out,
                                           moe_dtype out_dt, void* out_scales, hipStream_t stream) {
  MOE_CHECK(L > 0 && N > 0 && K > 0 && rows_cap >= 0, MOE_ERR_INVALID_ARG);
  MOE_CHECK(moe_host::valid_dtype(out_dt) && (epi == MOE_EPI_STORE_G || epi == MOE_EPI_SILU_MUL), MOE_ERR_INVALID_ARG);
  const bool silu = epi == MOE_EPI_SILU_MUL, mx4 = out_dt == MOE_FP8_E4M3;
  MOE_CHECK(L <= kMaxExperts && N % (mx4 ? 64 : 32) == 0 && K % 128 == 0 && K <= 1 << 24 &&
                static_cast<int64_t>(N) * K <= 1ll << 31 && static_cast<int64_t>(L) * N * K < 1ll << 39 &&
                rows_cap <= 1 << 30 && (!mx4 || silu), MOE_ERR_UNSUPPORTED);
  MOE_CHECK((out_scales != nullptr) == mx4 || rows_cap == 0, MOE_ERR_INVALID_ARG);
  if (rows_cap == 0) return MOE_OK;
  MOE_CHECK(a && a_scales && codes_packed && scales_packed && counts && offsets && out, MOE_ERR_INVALID_ARG);
  MOE_CHECK(aligned(a, 16) && aligned(codes_packed, 16) && aligned(out, 16) && aligned(a_scales, 4) &&
                aligned(scales_packed, 4), MOE_ERR_INVALID_ARG);
  const GemmArgs p{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(a_scales),
                   static_cast<const uint8_t*>(codes_packed), static_cast<const uint8_t*>(scales_packed), counts, offsets,
                   L, rows_cap, N, K, out, static_cast<uint8_t*>(out_scales)};
  if (mx4) gemm_mx4_kernel<kSiluMx4><<<kGrid, kThreads, 0, stream>>>(p);
  else if (silu && out_dt == MOE_F32) gemm_mx4_kernel<kSiluF32><<<kGrid, kThreads, 0, stream>>>(p);
  else if (silu) gemm_mx4_kernel<kSiluBf16><<<kGrid, kThreads, 0, stream>>>(p);
  else if (out_dt == MOE_F32) gemm_mx4_kernel<kStoreF32><<<kGrid, kThreads, 0, stream>>>(p);
  else gemm_mx4_kernel<kStoreBf16><<<kGrid, kThreads, 0, stream>>>(p);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}
