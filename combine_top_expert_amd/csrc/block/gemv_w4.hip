// moe_pack_w4 and moe_grouped_gemv_w4: the experts' products with 4-bit
// weights, for few rows per expert.
//
// G[q,n] = sum_g scale[n,g] sum_{k in g} A[q,k] value(code[n,k]).  The 4-bit
// values are exact in bf16 and go to the bf16 matrix cores (16 weight rows x 32
// columns), with up to 16 activation rows as the other operand.  Each scale
// group starts from a fresh accumulator, whose result is folded into fp32 sums
// with its scales.
//
// INT4 codes become 16 + code by placing the nibble in the mantissa of 16.0
// (7 instructions for 8 values); a product with the constant -24 over the same
// columns, shared by all of a wave's weight tiles, takes the offset off.  16 is
// the smallest offset that keeps a nibble in one binade, and keeps the cancelled
// part within about six times a group's own terms.
// E2M1 codes are converted by the hardware, two per instruction.
//
// Bound by reading the weights.  A workgroup's four waves share 64 weight rows
// (four 16-row tiles) and split the columns in stages of 128; each streams its
// share of the packed weights with 1 KB loads, and their sums meet in LDS.
//
// Measured on one decode step (128 tokens, about 130 rows for 32 experts), us:
// gate/up 4096 x 7168 INT4, a scale per 128, FP8 rows (492 MB) 72 to 80, the
// same loads without the arithmetic 71.6; down 7168 x 2048 E2M1, a scale per
// 32, bf16 rows (262 MB) 41.8 to 43.4, loads alone 41.1.  The same number of rows
// in every expert, 1 / 4 / 16 / 17 / 32 / 64 / 256: INT4 gate/up, FP8 rows 84 / 83 /
// 102 / 121 / 155 / 305 / 1203; bf16 rows 75 / 77 / 99 / 113 / 140 / 272 / 1088; E2M1
// gate/up, a scale per 128, FP8 rows 79 / 80 / 100 / 116 / 153 / 299 / 1178; per 32, bf16
// rows 81 / 84 / 105 / 119 / 148 / 291 / 1140; down 45 / 46 / 54 / 65 / 76 / 147 / 575.
// Past 32 rows the weights are read again for each 32.

#include <type_traits>

#include "block_common.h"

namespace {

using namespace moe_block;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kSimds = 1024;                    // of an MI355X
constexpr int kMaxWaves = 8;                    // of a workgroup
constexpr int kTiles = 4;                       // 16-row weight tiles of a wave

// ---------------------------------------------------------------- packing

// One thread makes one 16-byte piece: row l & 15 of the tile, four dwords of
// eight columns.  The column order inside a dword is the format's own.
__global__ __launch_bounds__(256) void pack_codes_kernel(const uint8_t* __restrict__ codes, int64_t pieces, int N,
                                                         int K, int fmt, uint4* __restrict__ out) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < pieces; i += gridDim.x * 256ll) {
    const int l = static_cast<int>(i & 63);
    const int64_t blk = i >> 6;
    const int ks = static_cast<int>(blk % (K / 128));
    const int64_t nt = blk / (K / 128);           // (expert, row tile)
    const uint8_t* row = codes + (nt * 16 + (l & 15)) * static_cast<int64_t>(K / 2) + ks * 64 + (l >> 4) * 4;
    uint32_t d[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint32_t v = *reinterpret_cast<const uint32_t*>(row + s * 16);
      if (fmt == MOE_W4_INT4) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w |= ((v >> (8 * j)) & 15u) << (4 * j) | ((v >> (8 * j + 4)) & 15u) << (4 * j + 16);
        v = (w << 3) | (w >> 29);
      }
      d[s] = v;
    }
    out[i] = make_uint4(d[0], d[1], d[2], d[3]);
  }
}

template <typename TS>
__global__ __launch_bounds__(256) void pack_scales_kernel(const TS* __restrict__ scales, int64_t count, int K, int group,
                                                          TS* __restrict__ out) {
  const int G = K / group, per = 128 / group;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < count; i += gridDim.x * 256ll) {
    const int g = static_cast<int>(i % per);
    const int r = static_cast<int>(i / per & 15);
    const int64_t blk = i / per >> 4;             // (expert, row tile, stage)
    const int ks = static_cast<int>(blk % (K / 128));
    out[i] = scales[(blk / (K / 128) * 16 + r) * G + ks * per + g];
  }
}

// ---------------------------------------------------------------- products

__device__ __forceinline__ bf16x8 as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint4 v = make_uint4(a, b, c, d);
  return __builtin_bit_cast(bf16x8, v);
}

// The mask of an INT4 code's place in a vector register: an and-or takes one
// constant from the scalar side only, and would otherwise be two instructions.
__device__ __forceinline__ uint32_t code_mask() {
  uint32_t m = 0x00780078u;
  asm("" : "+v"(m));
  return m;
}
template <int FMT> __device__ __forceinline__ bf16x8 unpack(uint32_t v, uint32_t m) {
  if constexpr (FMT == MOE_W4_INT4) {
    constexpr uint32_t o = 0x41804180u;
    return as_bf16x8((v & m) | o, ((v >> 4) & m) | o, ((v >> 8) & m) | o, (((v >> 12) | (v << 20)) & m) | o);
  } else {
    return as_bf16x8(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 3)));
  }
}

// 8 activations of one row as the matrix cores take them; e4m3 codes convert
// exactly
__device__ __forceinline__ bf16x8 as_rows(const uint4& v) { return __builtin_bit_cast(bf16x8, v); }
__device__ __forceinline__ bf16x8 as_rows(const uint2& v) {
  return as_bf16x8(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.x, 1.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.x, 1.0f, true)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.y, 1.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.y, 1.0f, true)));
}

__device__ __forceinline__ uint32_t dword(const uint4& v, int d) {
  return d == 0 ? v.x : d == 1 ? v.y : d == 2 ? v.z : v.w;
}

// SG neighbouring scales as loaded
template <typename TS, int SG> struct Scales {
  TS v[SG];
  __device__ __forceinline__ float get(int g) const {
    if constexpr (sizeof(TS) == 4) return v[g];
    else return __uint_as_float(static_cast<uint32_t>(v[g]) << 16);
  }
};
template <> struct Scales<uint16_t, 2> {
  uint32_t v;
  __device__ __forceinline__ float get(int g) const { return __uint_as_float(g ? v & 0xffff0000u : v << 16); }
};
template <> struct Scales<uint16_t, 4> {
  uint2 v;
  __device__ __forceinline__ float get(int g) const {
    const uint32_t w = g < 2 ? v.x : v.y;
    return __uint_as_float(g & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <> struct Scales<float, 2> {
  float2 v;
  __device__ __forceinline__ float get(int g) const { return g ? v.y : v.x; }
};
template <> struct Scales<float, 4> {
  float4 v;
  __device__ __forceinline__ float get(int g) const { return g == 0 ? v.x : g == 1 ? v.y : g == 2 ? v.z : v.w; }
};

// the value that lane LANE of this lane's 16-lane row holds
template <int LANE> __device__ __forceinline__ float row_bcast(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + LANE, 0xF, 0xF, true));
}

struct GemvArgs {
  const uint8_t* a;
  const float* a_scales;
  const uint8_t* codes;
  const void* scales;
  const int32_t* counts;
  const int32_t* offsets;
  int64_t rows_cap;
  int N, K;
  int waves;                                    // of a workgroup
  int split;                                    // waves that share a column block's stages
  int silu, out_f32;
  void* out;
};

constexpr int kPad = 4;                         // LDS row padding, floats
constexpr int kRedStride = kTiles * 16 + kPad;

// One column block (four weight tiles) of one expert for one wave, bf16 rows.
//
// Activations are the products' first operand and weights the second: lane
// 16 j + n then holds, of every 16 x 16 result, weight row n and activation rows
// 4 j .. 4 j + 3, and needs one scale per tile and group for its four values.
template <int FMT, typename TS, int SG, int MT> struct BlockBf16 {
  static constexpr int SPG = 4 / SG;            // 32-column steps of a scale group

  struct Rows {                                 // a stage's activations as loaded
    uint4 act[MT][4];
  };
  struct Weights {                              // a stage's weights
    uint4 w[kTiles];
  };
  struct Sc {                                   // and their scales
    Scales<TS, SG> s[kTiles];
  };
  // Up to 16 rows, everything is fetched one stage ahead (weights three stages
  // ahead at two waves per SIMD: the same time to 1 % for one or four rows, 2 to
  // 8 % more on the down shape); 32 rows leave no registers for the activations
  // and scales (168 at three waves per SIMD), which are fetched when their stage
  // begins; so are more than 8 bytes of scales a tile (INT4, whose offset takes
  // registers too: more than one scale; with four fp32 scales it spills two).
  static constexpr bool kAhead = MT == 1;
  static constexpr bool kScalesAhead = kAhead && (FMT == MOE_W4_INT4 ? SG == 1 : sizeof(Scales<TS, SG>) <= 8);

  // Addresses are a base that is the same for the wave plus 32 bits per lane:
  // one register a lane and no arithmetic per load.
  const uint8_t* w[kTiles];
  const TS* sc[kTiles];
  const uint8_t* a;
  uint32_t aoff[MT], scoff, lane16, mask;
  int KS, lane;
  f32x4 acc[kTiles][MT];

  __device__ __forceinline__ void load_rows(Rows& r, int ks) const {
    const uint8_t* at = a + static_cast<int64_t>(ks) * 256;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int s = 0; s < 4; ++s) r.act[m][s] = *reinterpret_cast<const uint4*>(at + aoff[m] + s * 64);
    }
  }
  __device__ __forceinline__ void load_scales(Sc& c, int ks) const {
#pragma unroll
    for (int f = 0; f < kTiles; ++f)
      c.s[f] = *reinterpret_cast<const Scales<TS, SG>*>(
          reinterpret_cast<const uint8_t*>(sc[f] + static_cast<int64_t>(ks) * (16 * SG)) + scoff);
  }
  __device__ __forceinline__ void load(Weights& b, int ks) const {
#pragma unroll
    for (int f = 0; f < kTiles; ++f) b.w[f] = moe::load_nt16(w[f] + static_cast<int64_t>(ks) * 1024 + lane16);
  }

  __device__ __forceinline__ void fold(int f, int m, float s, const f32x4& c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[f][m][i] = fmaf(c[i], s, acc[f][m][i]);
  }

  __device__ __forceinline__ void stage(const Weights& b, const Sc& sc, const Rows& r) {
#pragma unroll
    for (int g = 0; g < SG; ++g) {
      f32x4 c0[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        c0[m] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (FMT == MOE_W4_INT4) {
          const bf16x8 minus24 = as_bf16x8(0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u);
#pragma unroll
          for (int s = 0; s < SPG; ++s)
            c0[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_rows(r.act[m][g * SPG + s]), minus24, c0[m], 0, 0, 0);
        }
      }
      if constexpr (MT == 1) {
        // the four tiles side by side: four independent chains of products
        f32x4 c[kTiles] = {c0[0], c0[0], c0[0], c0[0]};
#pragma unroll
        for (int s = 0; s < SPG; ++s)
#pragma unroll
          for (int f = 0; f < kTiles; ++f)
            c[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_rows(r.act[0][g * SPG + s]),
                                                           unpack<FMT>(dword(b.w[f], g * SPG + s), mask), c[f], 0, 0, 0);
#pragma unroll
        for (int f = 0; f < kTiles; ++f) fold(f, 0, sc.s[f].get(g), c[f]);
      } else {
#pragma unroll
        for (int f = 0; f < kTiles; ++f) {
          f32x4 c[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) c[m] = c0[m];
#pragma unroll
          for (int s = 0; s < SPG; ++s) {
            const bf16x8 v = unpack<FMT>(dword(b.w[f], g * SPG + s), mask);
#pragma unroll
            for (int m = 0; m < MT; ++m)
              c[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_rows(r.act[m][g * SPG + s]), v, c[m], 0, 0, 0);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) fold(f, m, sc.s[f].get(g), c[m]);
          __builtin_amdgcn_sched_barrier(0);      // one tile's products at a time
        }
      }
    }
  }

  // Step U of the unrolled pair: the next stage's loads, then this stage.
  // Loads return in order, so those that are needed sooner go first.
  template <int U>
  __device__ __forceinline__ void step(int ks, int next, Weights (&b)[2], Sc (&c)[2], Rows (&r)[2]) {
    if (ks >= KS) return;
    constexpr int N = U ^ 1;
    if constexpr (!kScalesAhead) load_scales(c[0], ks);
    if constexpr (!kAhead) load_rows(r[0], ks);
    if (next < KS) {
      if constexpr (kScalesAhead) load_scales(c[N], next);
      if constexpr (kAhead) load_rows(r[N], next);
    }
    if (next < KS) load(b[N], next);
    __builtin_amdgcn_sched_barrier(0);
    stage(b[U], c[kScalesAhead ? U : 0], r[kAhead ? U : 0]);
  }

  // The sums of rows row0 .. row0 + rows - 1 (rows <= 16 MT) over the wave's
  // share of the stages: part, part + split, ...
  __device__ __forceinline__ void products(const GemvArgs& p, int e, int nb, int part, int64_t row0, int rows) {
    lane = moe::lane_id();
    const int n = lane & 15, j = lane >> 4;
    KS = p.K / 128;
    lane16 = lane * 16;
    mask = code_mask();
    scoff = n * SG * sizeof(TS);
#pragma unroll
    for (int f = 0; f < kTiles; ++f) {
      // 64 rows of G, or 32 gate rows and the 32 up rows they pair with
      const int64_t tile = static_cast<int64_t>(e) * (p.N / 16) +
                           (p.silu ? (f >> 1) * (p.N / 32) + nb * 2 + (f & 1) : nb * 4 + f);
      w[f] = p.codes + tile * KS * 1024;
      sc[f] = static_cast<const TS*>(p.scales) + tile * KS * (16 * SG);
    }
    a = p.a + row0 * p.K * 2;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      // lanes past the last row read row 0 again; what they compute is not stored
      const uint32_t r = m * 16 + n < rows ? m * 16 + n : 0;
      aoff[m] = (r * p.K + j * 8) * 2;
#pragma unroll
      for (int f = 0; f < kTiles; ++f) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (part >= KS) return;
    Weights b[2];
    Sc c[2];
    Rows r[2];
    if constexpr (kScalesAhead) load_scales(c[0], part);
    if constexpr (kAhead) load_rows(r[0], part);
    load(b[0], part);
    for (int ks = part; ks < KS; ks += 2 * p.split) {
      step<0>(ks, ks + p.split, b, c, r);
      step<1>(ks + p.split, ks + 2 * p.split, b, c, r);
    }
  }

  // this wave's 16 x 64 sums of activation rows 16 m .. into LDS rows
  __device__ __forceinline__ void spill(int m, float* rows16) const {
    const int n = lane & 15, j = lane >> 4;
#pragma unroll
    for (int f = 0; f < kTiles; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) rows16[(j * 4 + i) * kRedStride + f * 16 + n] = acc[f][m][i];
  }
};

// The same for FP8 rows.  Their scales are per activation row and stage, so
// weights are the first operand here: a lane then has one activation row and
// one such scale, and it is the weights' scales that lanes share.
//
// Lane 16 j + n holds, of every 16 x 16 result, weight rows 4 j .. 4 j + 3 and
// activation row n, so all 16 lanes of a row of lanes need the same scales.
// They share one load: lane n fetches the four scales of tile n & 3 and of the
// (n >> 2)-th group from here on, and the folds read them by row broadcasts,
// which are operand modifiers of the multiply-add.
template <int FMT, typename TS, int SG, int MT> struct BlockFp8 {
  static constexpr int SPG = 4 / SG;            // 32-column steps of a scale group
  static constexpr int CH = 4 / SG;             // stages that one scale load covers
  static constexpr int UN = CH < 2 ? 2 : CH;    // stages of the unrolled loop

  // Up to 16 rows, a stage's weights and activations are fetched one stage
  // ahead (weights three stages ahead at two waves per SIMD: the same time to
  // 1 % for one or four rows, 2 to 8 % more on the down shape); 32 rows leave
  // no registers for the activations (168 at three waves per SIMD), which are
  // fetched when their stage begins, and so are the scales where one load
  // covers four stages (two registers spilled there cost 6 us of 88 at L 32,
  // 4096 x 7168, in the 16-row path that does not use them).
  static constexpr bool kAhead = MT == 1;
  static constexpr bool kScalesAhead = kAhead || CH < 4;
  struct Rows {
    uint2 act[MT][4];
    float as[MT];
  };
  struct Buf {                                  // one stage's weights
    uint4 w[kTiles];
  };

  // Addresses are a base that is the same for the wave plus 32 bits per lane:
  // one register a lane and no arithmetic per load.
  const uint8_t* w[kTiles];
  const uint8_t* a;
  const float* as;
  const TS* sc;
  uint32_t aoff[MT], asoff[MT], scoff, lane16, mask;
  int KS, usub, lane;
  f32x4 acc[kTiles][MT];

  __device__ __forceinline__ void load_rows(Rows& r, int ks) const {
    const uint8_t* at = a + static_cast<int64_t>(ks) * 128;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int s = 0; s < 4; ++s) r.act[m][s] = *reinterpret_cast<const uint2*>(at + aoff[m] + s * 32);
      r.as[m] = *reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(as + ks) + asoff[m]);
    }
  }
  __device__ __forceinline__ void load(Buf& b, int ks) const {
#pragma unroll
    for (int f = 0; f < kTiles; ++f) b.w[f] = moe::load_nt16(w[f] + static_cast<int64_t>(ks) * 1024 + lane16);
  }
  __device__ __forceinline__ f32x4 scales(int ks) const {
    const uint32_t k = min(ks + usub, KS - 1);
    const uint8_t* base = reinterpret_cast<const uint8_t*>(sc);
    const uint32_t at = scoff + k * (SG * 16 * static_cast<uint32_t>(sizeof(TS)));
    if constexpr (SG == 1 && sizeof(TS) == 4) return *reinterpret_cast<const f32x4*>(base + at);
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const TS* one = reinterpret_cast<const TS*>(base + (at + i * SG * static_cast<uint32_t>(sizeof(TS))));
      if constexpr (sizeof(TS) == 4) v[i] = *one;
      else v[i] = __uint_as_float(static_cast<uint32_t>(*one) << 16);
    }
    return v;
  }

  template <int SUB, int G, int F> __device__ __forceinline__ void fold(const f32x4& sc, const Rows& r, int m, const f32x4& c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = row_bcast<(SUB * SG + G) * 4 + F>(sc[i]);
      acc[F][m][i] = fmaf(c[i], s * r.as[m], acc[F][m][i]);
    }
  }

  template <int SUB, int G> __device__ __forceinline__ void group(const f32x4& sc, const Buf& b, const Rows& r) {
    f32x4 c0[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      c0[m] = f32x4{0.f, 0.f, 0.f, 0.f};
      if constexpr (FMT == MOE_W4_INT4) {
        const bf16x8 minus24 = as_bf16x8(0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u);
#pragma unroll
        for (int s = 0; s < SPG; ++s)
          c0[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(minus24, as_rows(r.act[m][G * SPG + s]), c0[m], 0, 0, 0);
      }
    }
    if constexpr (MT == 1) {
      // the four tiles side by side: four independent chains of products
      f32x4 c[kTiles] = {c0[0], c0[0], c0[0], c0[0]};
#pragma unroll
      for (int s = 0; s < SPG; ++s)
#pragma unroll
        for (int f = 0; f < kTiles; ++f)
          c[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(unpack<FMT>(dword(b.w[f], G * SPG + s), mask),
                                                         as_rows(r.act[0][G * SPG + s]), c[f], 0, 0, 0);
      fold<SUB, G, 0>(sc, r, 0, c[0]);
      fold<SUB, G, 1>(sc, r, 0, c[1]);
      fold<SUB, G, 2>(sc, r, 0, c[2]);
      fold<SUB, G, 3>(sc, r, 0, c[3]);
    } else {
      tile<SUB, G, 0>(sc, b, r, c0);
      tile<SUB, G, 1>(sc, b, r, c0);
      tile<SUB, G, 2>(sc, b, r, c0);
      tile<SUB, G, 3>(sc, b, r, c0);
    }
  }
  template <int SUB, int G, int F>
  __device__ __forceinline__ void tile(const f32x4& shared, const Buf& b, const Rows& r, const f32x4 (&c0)[MT]) {
    f32x4 sc = shared;
    // The compiler makes a stage's 64 broadcasts of loaded fp32 scales at its
    // beginning and spills 180 registers, unless they become values of the tile;
    // bf16 scales, which are converted first, it leaves where they are.
    if constexpr (sizeof(TS) == 4) asm volatile("" : "+v"(sc[0]), "+v"(sc[1]), "+v"(sc[2]), "+v"(sc[3]));
    f32x4 c[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) c[m] = c0[m];
#pragma unroll
    for (int s = 0; s < SPG; ++s) {
      const bf16x8 v = unpack<FMT>(dword(b.w[F], G * SPG + s), mask);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        c[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, as_rows(r.act[m][G * SPG + s]), c[m], 0, 0, 0);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) fold<SUB, G, F>(sc, r, m, c[m]);
    __builtin_amdgcn_sched_barrier(0);          // one tile's products at a time
  }

  template <int SUB> __device__ __forceinline__ void stage(const f32x4& sc, const Buf& b, const Rows& r) {
    group<SUB, 0>(sc, b, r);
    if constexpr (SG >= 2) group<SUB, 1>(sc, b, r);
    if constexpr (SG == 4) {
      group<SUB, 2>(sc, b, r);
      group<SUB, 3>(sc, b, r);
    }
  }

  // Step U of the unrolled loop: the next stage's loads, then this stage.
  // Loads return in order, so those that are needed sooner go first.
  template <int U, typename KsOf>
  __device__ __forceinline__ void step(int i, int n, const KsOf& ks_of, f32x4& sc, f32x4& sc_next, Buf (&b)[2],
                                       Rows (&r)[2]) {
    if (i >= n) return;
    if constexpr (U % CH == 0) {
      if constexpr (kScalesAhead) {
        sc = sc_next;
        if (i + CH < n) sc_next = scales(ks_of(i + CH));
      } else {
        sc = scales(ks_of(i));
      }
    }
    if constexpr (kAhead) {
      if (i + 1 < n) load_rows(r[(U + 1) & 1], ks_of(i + 1));
    } else {
      load_rows(r[0], ks_of(i));
    }
    if (i + 1 < n) load(b[(U + 1) & 1], ks_of(i + 1));
    __builtin_amdgcn_sched_barrier(0);
    stage<U % CH>(sc, b[U & 1], r[kAhead ? U & 1 : 0]);
  }

  // The sums of rows row0 .. row0 + rows - 1 (rows <= 16 MT) over the wave's
  // share of the stages: chunks part, part + split, ... of CH stages.
  __device__ __forceinline__ void products(const GemvArgs& p, int e, int nb, int part, int64_t row0, int rows) {
    lane = moe::lane_id();
    const int n = lane & 15, j = lane >> 4;
    KS = p.K / 128;
    auto tile = [&](int f) {   // 64 rows of G, or 32 gate rows and the 32 up rows they pair with
      return static_cast<int64_t>(e) * (p.N / 16) + (p.silu ? (f >> 1) * (p.N / 32) + nb * 2 + (f & 1) : nb * 4 + f);
    };
#pragma unroll
    for (int f = 0; f < kTiles; ++f) w[f] = p.codes + tile(f) * KS * 1024;
    lane16 = lane * 16;
    mask = code_mask();
    const int u = n >> 2;
    usub = u / SG;
    sc = static_cast<const TS*>(p.scales) + tile(0) * KS * SG * 16;
    scoff = static_cast<uint32_t>((tile(n & 3) - tile(0)) * KS * SG * 16 + j * 4 * SG + u % SG) * sizeof(TS);
    a = p.a + row0 * p.K;
    as = p.a_scales + row0 * KS;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      // lanes past the last row read row 0 again; what they compute is not stored
      const uint32_t r = m * 16 + n < rows ? m * 16 + n : 0;
      aoff[m] = r * p.K + j * 8;
      asoff[m] = r * KS * 4;
#pragma unroll
      for (int f = 0; f < kTiles; ++f) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int NC = (KS + CH - 1) / CH;
    const int own = part < NC ? (NC - part + p.split - 1) / p.split : 0;
    const bool last = own > 0 && (own - 1) * p.split + part == NC - 1;
    const int count = own * CH - (last ? NC * CH - KS : 0);
    auto ks_of = [&](int i) { return ((i / CH) * p.split + part) * CH + i % CH; };
    if (count == 0) return;
    Buf b[2];
    Rows r[2];
    f32x4 sc, sc_next = scales(ks_of(0));
    if constexpr (kAhead) load_rows(r[0], ks_of(0));
    load(b[0], ks_of(0));
    for (int i = 0; i < count; i += UN) {
      step<0>(i, count, ks_of, sc, sc_next, b, r);
      step<1>(i + 1, count, ks_of, sc, sc_next, b, r);
      if constexpr (UN == 4) {
        step<2>(i + 2, count, ks_of, sc, sc_next, b, r);
        step<3>(i + 3, count, ks_of, sc, sc_next, b, r);
      }
    }
  }

  __device__ __forceinline__ void spill(int m, float* rows16) const {
    const int n = lane & 15, j = lane >> 4;
#pragma unroll
    for (int f = 0; f < kTiles; ++f) *reinterpret_cast<f32x4*>(rows16 + n * kRedStride + f * 16 + j * 4) = acc[f][m];
  }
};

// The waves' sums through LDS, in wave order, 16 rows at a time, and the
// epilogue.  With split 1 a wave only meets itself.
template <int MT, typename B>
__device__ __forceinline__ void store(const B& blk, const GemvArgs& p, int nb, int part, int64_t row0, int rows, float* mine) {
  const int lane = blk.lane;
  const int cols = p.silu ? 32 : 64, quads = cols / 4;
  const int ldo = p.silu ? p.N / 2 : p.N;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (p.split > 1) __syncthreads();
    blk.spill(m, mine + part * 16 * kRedStride);
    if (p.split > 1) __syncthreads();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int i = part * MOE_WAVE + lane; i < 16 * quads; i += p.split * MOE_WAVE) {
      const int r = i / quads, q = i % quads * 4;
      if (m * 16 + r >= rows) break;
      f32x4 v = {0.f, 0.f, 0.f, 0.f}, u = v;
      for (int s = 0; s < p.split; ++s) {
        const float* src = mine + (s * 16 + r) * kRedStride + q;
        v += *reinterpret_cast<const f32x4*>(src);
        if (p.silu) u += *reinterpret_cast<const f32x4*>(src + 32);
      }
      if (p.silu) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = moe::silu(v[k]) * u[k];
      }
      const int64_t at = (row0 + m * 16 + r) * ldo + nb * cols + q;
      if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <int FMT, bool FP8, typename TS, int SG, int MT>
using Block = std::conditional_t<FP8, BlockFp8<FMT, TS, SG, MT>, BlockBf16<FMT, TS, SG, MT>>;

template <int FMT, bool FP8, typename TS, int SG>
__global__ __launch_bounds__(kMaxWaves * MOE_WAVE, 3) void gemv_w4_kernel(GemvArgs p) {
  extern __shared__ float red[];                            // [waves][16][kRedStride]
  const int nbs = p.N / 64, blocks = p.waves / p.split;      // column blocks of an expert, of this workgroup
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / p.split, part = wave % p.split;
  const int per = (nbs + blocks - 1) / blocks;
  const int e = blockIdx.x / per, nb = (blockIdx.x % per) * blocks + group;
  // nb is the same for all waves that meet at a barrier
  const int64_t off = p.offsets[e];
  int64_t rows = p.counts[e];
  if (off < 0 || nb >= nbs) return;
  if (rows > p.rows_cap - off) rows = p.rows_cap - off;
  float* mine = red + group * p.split * 16 * kRedStride;
  for (int64_t r = 0; r < rows; r += 32) {
    const int m = static_cast<int>(rows - r < 32 ? rows - r : 32);
    if (m <= 16) {
      Block<FMT, FP8, TS, SG, 1> w;
      w.products(p, e, nb, part, off + r, m);
      store<1>(w, p, nb, part, off + r, m, mine);
    } else {
      Block<FMT, FP8, TS, SG, 2> w;
      w.products(p, e, nb, part, off + r, m);
      store<2>(w, p, nb, part, off + r, m, mine);
    }
  }
}

// How many waves share a column block: up to four while each keeps eight
// stages (a wave's first loads and the sums' meeting cost about four stages'
// time), and up to eight with four stages each where the blocks would not fill
// the card's SIMDs once.  Measured with four rows an expert, INT4 with a scale per
// 128, in us, for 1 / 2 / 4 / 8 waves, FP8 rows and bf16 rows: L 32, 4096 x 7168: 81 / 84 /
// 82 / 102 and 79 / 80 / 77 / 92; L 32, 7168 x 2048: 54 / 46 / 54 / 85 and 53 / 43 / 43 / 65; L
// 64, 4096 x 1408: 35 / 37 / 43 / 85 and 34 / 34 / 38 / 61; L 1, 4096 x 7168: 46 / 25 / 16 / 13
// and 41 / 23 / 14 / 12; L 1, 7168 x 2048: 15 / 10 / 7.2 / 7.4 and 14 / 9.3 / 6.6 / 6.2.
void pick_split(GemvArgs& p, int L) {
  const int KS = p.K / 128;
  const int64_t blocks = static_cast<int64_t>(L) * (p.N / 64);
  p.split = 1;
  while (p.split < 4 && KS >= 16 * p.split) p.split *= 2;
  while (p.split < kMaxWaves && KS >= 8 * p.split && blocks * p.split <= kSimds) p.split *= 2;
  p.waves = p.split > 4 ? p.split : 4;
}

template <int FMT, bool FP8, typename TS>
void launch_group(const GemvArgs& a, int L, int group, hipStream_t stream) {
  GemvArgs p = a;
  pick_split(p, L);
  const int nbs = p.N / 64, blocks = p.waves / p.split;
  const int grid = L * ((nbs + blocks - 1) / blocks), threads = p.waves * MOE_WAVE;
  const size_t lds = static_cast<size_t>(p.waves) * 16 * kRedStride * sizeof(float);
  if (group == 128) gemv_w4_kernel<FMT, FP8, TS, 1><<<grid, threads, lds, stream>>>(p);
  else if (group == 64) gemv_w4_kernel<FMT, FP8, TS, 2><<<grid, threads, lds, stream>>>(p);
  else gemv_w4_kernel<FMT, FP8, TS, 4><<<grid, threads, lds, stream>>>(p);
}
template <int FMT, bool FP8> void launch_scale(const GemvArgs& p, int L, bool s32, int group, hipStream_t stream) {
  if (s32) launch_group<FMT, FP8, float>(p, L, group, stream);
  else launch_group<FMT, FP8, uint16_t>(p, L, group, stream);
}

inline bool w4_sizes(int L, int N, int K) { return L >= 1 && N >= 1 && K >= 1; }
inline bool w4_limits(int L, int N, int K, int group) {
  return N % 128 == 0 && K % 128 == 0 && L <= 1024 && (group == 32 || group == 64 || group == 128) &&
         static_cast<int64_t>(N) * K <= (1ll << 31) && K <= (1 << 24);   // 32-bit offsets within an expert
}

}  // namespace

extern "C" moe_status moe_pack_w4(const void* codes, const void* scales, moe_dtype s_dt, moe_w4_format fmt, int L,
                                  int N, int K, int group, void* codes_packed, void* scales_packed,
                                  hipStream_t stream) {
  MOE_CHECK(w4_sizes(L, N, K), MOE_ERR_INVALID_ARG);
  MOE_CHECK(moe_host::valid_dtype(s_dt) && (fmt == MOE_W4_INT4 || fmt == MOE_W4_E2M1), MOE_ERR_INVALID_ARG);
  MOE_CHECK(real_dtype(s_dt) && w4_limits(L, N, K, group), MOE_ERR_UNSUPPORTED);
  MOE_CHECK(codes && scales && codes_packed && scales_packed && codes != codes_packed && scales != scales_packed,
            MOE_ERR_INVALID_ARG);
  MOE_CHECK(aligned16(codes) && aligned16(codes_packed) && aligned16(scales_packed), MOE_ERR_INVALID_ARG);
  const int64_t pieces = static_cast<int64_t>(L) * N * (K / 32);
  const int64_t count = static_cast<int64_t>(L) * N * (K / group);
  auto grid = [](int64_t n) { return static_cast<int>((n + 255) / 256 < 16384 ? (n + 255) / 256 : 16384); };
  pack_codes_kernel<<<grid(pieces), 256, 0, stream>>>(static_cast<const uint8_t*>(codes), pieces, N, K, fmt,
                                                      static_cast<uint4*>(codes_packed));
  MOE_LAUNCH_CHECK();
  if (s_dt == MOE_F32)
    pack_scales_kernel<<<grid(count), 256, 0, stream>>>(static_cast<const float*>(scales), count, K, group,
                                                        static_cast<float*>(scales_packed));
  else
    pack_scales_kernel<<<grid(count), 256, 0, stream>>>(static_cast<const uint16_t*>(scales), count, K, group,
                                                        static_cast<uint16_t*>(scales_packed));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

extern "C" moe_status moe_grouped_gemv_w4(const void* a, moe_dtype a_dt, const float* a_scales,
                                          const void* codes_packed, const void* scales_packed, moe_dtype s_dt,
                                          moe_w4_format fmt, int group, const int32_t* counts, const int32_t* offsets,
                                          int L, int64_t rows_cap, int N, int K, moe_w13_epilogue epi, void* out,
                                          moe_dtype out_dt, hipStream_t stream) {
  MOE_CHECK(w4_sizes(L, N, K) && rows_cap >= 0, MOE_ERR_INVALID_ARG);
  MOE_CHECK(moe_host::valid_dtype(a_dt) && moe_host::valid_dtype(s_dt) && moe_host::valid_dtype(out_dt),
            MOE_ERR_INVALID_ARG);
  MOE_CHECK((fmt == MOE_W4_INT4 || fmt == MOE_W4_E2M1) && (epi == MOE_EPI_STORE_G || epi == MOE_EPI_SILU_MUL),
            MOE_ERR_INVALID_ARG);
  MOE_CHECK(a_dt != MOE_F32 && real_dtype(s_dt) && real_dtype(out_dt), MOE_ERR_UNSUPPORTED);
  MOE_CHECK(w4_limits(L, N, K, group), MOE_ERR_UNSUPPORTED);
  // a launch has L N split lanes, and waves share a block's stages from K = 2048 on
  MOE_CHECK(static_cast<int64_t>(L) * N * K < 1ll << 39, MOE_ERR_UNSUPPORTED);
  if (rows_cap == 0) return MOE_OK;
  MOE_CHECK(a && codes_packed && scales_packed && counts && offsets && out, MOE_ERR_INVALID_ARG);
  MOE_CHECK(a_dt != MOE_FP8_E4M3 || a_scales, MOE_ERR_INVALID_ARG);
  MOE_CHECK(aligned16(a) && aligned16(codes_packed) && aligned16(scales_packed) && aligned16(out), MOE_ERR_INVALID_ARG);
  const GemvArgs p{static_cast<const uint8_t*>(a), a_scales, static_cast<const uint8_t*>(codes_packed), scales_packed,
                   counts, offsets, rows_cap, N, K, 4, 4, epi == MOE_EPI_SILU_MUL, out_dt == MOE_F32, out};
  const bool s32 = s_dt == MOE_F32;
  const bool fp8 = a_dt == MOE_FP8_E4M3;
  if (fmt == MOE_W4_INT4) {
    if (fp8) launch_scale<MOE_W4_INT4, true>(p, L, s32, group, stream);
    else launch_scale<MOE_W4_INT4, false>(p, L, s32, group, stream);
  } else {
    if (fp8) launch_scale<MOE_W4_E2M1, true>(p, L, s32, group, stream);
    else launch_scale<MOE_W4_E2M1, false>(p, L, s32, group, stream);
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}
