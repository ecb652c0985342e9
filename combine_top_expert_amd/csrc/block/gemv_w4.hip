// moe_pack_w4 and moe_grouped_gemv_w4: the experts' products with 4-bit
// weights, for few rows per expert.
//
// G[q,n] = sum_g scale[n,g] sum_{k in g} A[q,k] value(code[n,k]).  The 4-bit
// values are exact in bf16 and go to the bf16 matrix cores as the first
// operand (16 weight rows x 32 columns), up to 16 activation rows as the
// second; a lane's four results are then four neighbouring weight rows of one
// activation row.  Each scale group starts from a fresh accumulator, whose
// result is folded into fp32 sums with its scales.
//
// INT4 codes become 16 + code by placing the nibble in the mantissa of 16.0
// (one shift and one and-or per two values); a product with the constant -24
// over the same columns, shared by all of a wave's weight tiles, takes the
// offset off.  16 is the smallest offset that keeps a nibble in one binade,
// and keeps the cancelled part within about six times a group's own terms.
// E2M1 codes are converted by the hardware, two per instruction.
//
// Bound by reading the weights.  A workgroup's four waves share 64 weight rows
// (four 16-row tiles) and split the columns in stages of 128; each streams its
// share of the packed weights with 1 KB loads, and their sums meet in LDS.

#include "block_common.h"

namespace {

using namespace moe_block;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * MOE_WAVE;
constexpr int kTiles = 4;                       // 16-row weight tiles of a workgroup

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
        v = w;
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
    const int r = static_cast<int>(i & 15);
    const int g = static_cast<int>((i >> 4) % G);  // stage * per + group of the stage
    const int64_t nt = (i >> 4) / G;
    out[i] = scales[(nt * 16 + r) * G + g];
  }
}

// ---------------------------------------------------------------- products

__device__ __forceinline__ bf16x8 as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint4 v = make_uint4(a, b, c, d);
  return __builtin_bit_cast(bf16x8, v);
}

template <int FMT> __device__ __forceinline__ bf16x8 unpack(uint32_t v) {
  if constexpr (FMT == MOE_W4_INT4) {
    constexpr uint32_t m = 0x00780078u, o = 0x41804180u;
    return as_bf16x8(((v << 3) & m) | o, ((v >> 1) & m) | o, ((v >> 5) & m) | o, ((v >> 9) & m) | o);
  } else {
    return as_bf16x8(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 3)));
  }
}

// 8 activations of one row: bf16 as they are, e4m3 codes converted exactly
template <bool FP8> __device__ __forceinline__ bf16x8 load_act(const uint8_t* p) {
  if constexpr (!FP8) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(p));
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return as_bf16x8(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.x, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.x, 1.0f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.y, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.y, 1.0f, true)));
  }
}

template <typename TS> __device__ __forceinline__ f32x4 load_scales(const TS* p);
template <> __device__ __forceinline__ f32x4 load_scales<float>(const float* p) {
  return *reinterpret_cast<const f32x4*>(p);
}
template <> __device__ __forceinline__ f32x4 load_scales<uint16_t>(const uint16_t* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return f32x4{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
               __uint_as_float(v.y & 0xffff0000u)};
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
  void* out;
  int out_f32;
};

constexpr int kPad = 4;                                   // LDS row padding, floats
constexpr int kRedStride = kTiles * 16 + kPad;

// One block of at most 16 * MT rows against the workgroup's 64 weight rows.
template <int FMT, bool FP8, typename TS, int SG, bool SILU, int MT>
__device__ __forceinline__ void rows_block(const GemvArgs& p, int e, int nb, int64_t row0, int rows, float* red) {
  const int lane = moe::lane_id(), wave = threadIdx.x >> 6;
  const int n = lane & 15, j = lane >> 4;
  const int KS = p.K / 128;
  constexpr int ESZ = FP8 ? 1 : 2;
  // the workgroup's tiles: 64 rows of G, or 32 gate and the 32 up rows they pair with
  int64_t tile[kTiles];
#pragma unroll
  for (int f = 0; f < kTiles; ++f) {
    const int64_t base = static_cast<int64_t>(e) * (p.N / 16);
    tile[f] = SILU ? base + (f >> 1) * (p.N / 32) + nb * 2 + (f & 1) : base + nb * 4 + f;
  }
  const TS* scales = static_cast<const TS*>(p.scales);
  f32x4 acc[kTiles][MT];
#pragma unroll
  for (int f = 0; f < kTiles; ++f)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};

  const bf16x8 minus24 = as_bf16x8(0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u);
  constexpr int SPG = 4 / SG;                              // 32-column steps per group
  for (int ks = wave; ks < KS; ks += kWaves) {
    uint4 w[kTiles];
    f32x4 sc[kTiles][SG];
#pragma unroll
    for (int f = 0; f < kTiles; ++f) {
      w[f] = *reinterpret_cast<const uint4*>(p.codes + ((tile[f] * KS + ks) * 64 + lane) * 16);
#pragma unroll
      for (int g = 0; g < SG; ++g) sc[f][g] = load_scales<TS>(scales + ((tile[f] * KS + ks) * SG + g) * 16 + j * 4);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = m * 16 + n;
      const bool live = r < rows;
      const uint8_t* ap = p.a + ((row0 + r) * p.K + ks * 128 + j * 8) * ESZ;
      bf16x8 act[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) act[s] = live ? load_act<FP8>(ap + s * 32 * ESZ) : as_bf16x8(0, 0, 0, 0);
      const float as = FP8 ? (live ? p.a_scales[(row0 + r) * KS + ks] : 0.f) : 1.f;
#pragma unroll
      for (int g = 0; g < SG; ++g) {
        f32x4 c0 = {0.f, 0.f, 0.f, 0.f};
        if constexpr (FMT == MOE_W4_INT4) {
#pragma unroll
          for (int s = 0; s < SPG; ++s)
            c0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(minus24, act[g * SPG + s], c0, 0, 0, 0);
        }
#pragma unroll
        for (int f = 0; f < kTiles; ++f) {
          const uint32_t d[4] = {w[f].x, w[f].y, w[f].z, w[f].w};
          f32x4 c = c0;
#pragma unroll
          for (int s = 0; s < SPG; ++s)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(unpack<FMT>(d[g * SPG + s]), act[g * SPG + s], c, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[f][m][i] = fmaf(c[i], FP8 ? sc[f][g][i] * as : sc[f][g][i], acc[f][m][i]);
        }
      }
    }
  }

  // the four waves' sums, in wave order, 16 rows at a time
  constexpr int COLS = SILU ? 32 : 64;
  constexpr int QUADS = COLS / 4;
  const int ldo = SILU ? p.N / 2 : p.N;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    __syncthreads();
#pragma unroll
    for (int f = 0; f < kTiles; ++f)
      *reinterpret_cast<f32x4*>(red + (wave * 16 + n) * kRedStride + f * 16 + j * 4) = acc[f][m];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * QUADS; i += kThreads) {
      const int r = i / QUADS, q = i % QUADS * 4;
      if (m * 16 + r >= rows) continue;
      f32x4 v = {0.f, 0.f, 0.f, 0.f}, u = v;
#pragma unroll
      for (int s = 0; s < kWaves; ++s) {
        const float* src = red + (s * 16 + r) * kRedStride + q;
        v += *reinterpret_cast<const f32x4*>(src);
        if constexpr (SILU) u += *reinterpret_cast<const f32x4*>(src + 32);
      }
      if constexpr (SILU) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = moe::silu(v[k]) * u[k];
      }
      const int64_t at = (row0 + m * 16 + r) * ldo + nb * COLS + q;
      if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
  }
}

template <int FMT, bool FP8, typename TS, int SG, bool SILU>
__global__ __launch_bounds__(kThreads) void gemv_w4_kernel(GemvArgs p) {
  __shared__ float red[kWaves * 16 * kRedStride];
  const int nbs = p.N / 64;
  const int e = blockIdx.x / nbs, nb = blockIdx.x % nbs;
  const int64_t off = p.offsets[e];
  int64_t rows = p.counts[e];
  if (off < 0) return;
  if (rows > p.rows_cap - off) rows = p.rows_cap - off;
  for (int64_t r = 0; r < rows; r += 64) {
    const int m = static_cast<int>(rows - r < 64 ? rows - r : 64);
    if (m <= 16) rows_block<FMT, FP8, TS, SG, SILU, 1>(p, e, nb, off + r, m, red);
    else if (m <= 32) rows_block<FMT, FP8, TS, SG, SILU, 2>(p, e, nb, off + r, m, red);
    else rows_block<FMT, FP8, TS, SG, SILU, 4>(p, e, nb, off + r, m, red);
  }
}

template <int FMT, bool FP8, typename TS, int SG>
void launch_epi(const GemvArgs& p, int L, bool silu, hipStream_t stream) {
  const int grid = L * (p.N / 64);
  if (silu) gemv_w4_kernel<FMT, FP8, TS, SG, true><<<grid, kThreads, 0, stream>>>(p);
  else gemv_w4_kernel<FMT, FP8, TS, SG, false><<<grid, kThreads, 0, stream>>>(p);
}
template <int FMT, bool FP8, typename TS>
void launch_group(const GemvArgs& p, int L, int group, bool silu, hipStream_t stream) {
  if (group == 128) launch_epi<FMT, FP8, TS, 1>(p, L, silu, stream);
  else if (group == 64) launch_epi<FMT, FP8, TS, 2>(p, L, silu, stream);
  else launch_epi<FMT, FP8, TS, 4>(p, L, silu, stream);
}
template <int FMT, bool FP8>
void launch_scale(const GemvArgs& p, int L, bool s32, int group, bool silu, hipStream_t stream) {
  if (s32) launch_group<FMT, FP8, float>(p, L, group, silu, stream);
  else launch_group<FMT, FP8, uint16_t>(p, L, group, silu, stream);
}

inline bool w4_sizes(int L, int N, int K) { return L >= 1 && N >= 1 && K >= 1; }
inline bool w4_limits(int L, int N, int K, int group) {
  return N % 128 == 0 && K % 128 == 0 && L <= 1024 && (group == 32 || group == 64 || group == 128);
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
  MOE_CHECK(static_cast<int64_t>(L) * (N / 64) <= 0x7fffffff, MOE_ERR_UNSUPPORTED);
  if (rows_cap == 0) return MOE_OK;
  MOE_CHECK(a && codes_packed && scales_packed && counts && offsets && out, MOE_ERR_INVALID_ARG);
  MOE_CHECK(a_dt != MOE_FP8_E4M3 || a_scales, MOE_ERR_INVALID_ARG);
  MOE_CHECK(aligned16(a) && aligned16(codes_packed) && aligned16(scales_packed) && aligned16(out), MOE_ERR_INVALID_ARG);
  const GemvArgs p{static_cast<const uint8_t*>(a), a_scales, static_cast<const uint8_t*>(codes_packed), scales_packed,
                   counts, offsets, rows_cap, N, K, out, out_dt == MOE_F32};
  const bool silu = epi == MOE_EPI_SILU_MUL, s32 = s_dt == MOE_F32;
  const bool fp8 = a_dt == MOE_FP8_E4M3;
  if (fmt == MOE_W4_INT4) {
    if (fp8) launch_scale<MOE_W4_INT4, true>(p, L, s32, group, silu, stream);
    else launch_scale<MOE_W4_INT4, false>(p, L, s32, group, silu, stream);
  } else {
    if (fp8) launch_scale<MOE_W4_E2M1, true>(p, L, s32, group, silu, stream);
    else launch_scale<MOE_W4_E2M1, false>(p, L, s32, group, silu, stream);
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}
