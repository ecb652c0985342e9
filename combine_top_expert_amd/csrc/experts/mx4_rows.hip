// moe_quantize_mx4, moe_permute_mx4 and moe_pack_mx4: rows and weights to
// microscaled 4 bits, and weights into the products' order.
//
// A block is 32 neighbouring columns: its largest magnitude gives the power of
// two, and x / 2^e is exact, so a code is one rounding of x itself.  A lane loads
// 16 bytes, so that each load of a wave is one contiguous KB; the lanes of a
// block (4 with bf16, 8 with fp32) meet in DPP moves.
//
// Bound by memory: the bytes of x, and 17/32 of a byte a value back.  470 M bf16
// values (1.19 GB) take 191 us, 6.2 TB/s; dispatch of 8192 tokens of 7168 bf16 columns to 32 of 256 experts
// (3300 of them have one: 63 MB, which the 256 MB cache holds) 12.2 to 13.5 us, of 128 tokens 2.8 us, a launch.

#include "experts_common.h"

namespace {

using namespace moe_experts;

// A lane's 16 bytes of x, as fp32
template <typename T> struct Piece;
template <> struct Piece<uint16_t> {                 // bf16
  static constexpr int kValues = 8;
  float v[8];
  __device__ __forceinline__ explicit Piece(const uint4& r) {
    const uint32_t d[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(d[i] << 16);
      v[2 * i + 1] = __uint_as_float(d[i] & 0xffff0000u);
    }
  }
};
template <> struct Piece<float> {
  static constexpr int kValues = 4;
  float v[4];
  __device__ __forceinline__ explicit Piece(const uint4& r)
      : v{__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w)} {}
};

// A lane's codes (32 bits of bf16, 16 of fp32 rows) and its block's scale
template <typename T> __device__ __forceinline__ void quantise(const uint4& raw, uint32_t& codes, uint32_t& scale) {
  const Piece<T> p(raw);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < Piece<T>::kValues; ++i) top = max(top, magnitude(p.v[i]));
  top = dpp_max<kXor2>(dpp_max<kXor1>(top));
  if constexpr (sizeof(T) == 4) top = dpp_max<kHalfMirror>(top);
  scale = mx4_scale(top);
  if constexpr (sizeof(T) == 2) codes = mx4_codes8(p.v, scale);
  else codes = mx4_codes4(p.v, scale);
}

// A lane's 16 bytes of what its codes stand for.  e2m1 times a power of two is
// exact in bf16 (2 bits, 8-bit exponent, subnormals down to 2^-133).
template <typename T> __device__ __forceinline__ uint4 values_of(uint32_t codes, uint32_t scale) {
  uint32_t d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      d[i] = __float_as_uint(mx4_value(codes >> (4 * i), scale));
    } else {
      d[i] = __float_as_uint(mx4_value(codes >> (8 * i), scale)) >> 16 |
             (__float_as_uint(mx4_value(codes >> (8 * i + 4), scale)) & 0xffff0000u);
    }
  }
  return make_uint4(d[0], d[1], d[2], d[3]);
}

constexpr int kChunks = 4;                       // 16-byte loads of a lane

// x is one run of blocks (rows are dense and a multiple of 32 columns).  A wave
// takes 4 chunks of 1 KB.  With bf16 the four lanes of a block exchange their
// codes so that lane q of them holds the whole block of chunk q: one 16-byte
// store of codes and one byte of scale a lane for everything the wave loaded.
// With fp32, pairs of lanes join their 16-bit halves.
template <typename T, bool VALUES>
__global__ __launch_bounds__(256) void quantize_kernel(const uint4* __restrict__ x, int64_t pieces,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                       uint4* __restrict__ values) {
  const int lane = moe::lane_id();
  const int64_t first = (blockIdx.x * 4ll + (threadIdx.x >> 6)) * (kChunks * MOE_WAVE);
  uint4 raw[kChunks];
#pragma unroll
  for (int u = 0; u < kChunks; ++u) {
    const int64_t i = first + u * MOE_WAVE + lane;
    raw[u] = i < pieces ? moe::load_nt16(x + i) : make_uint4(0, 0, 0, 0);
  }
  uint32_t c[kChunks], s[kChunks];
#pragma unroll
  for (int u = 0; u < kChunks; ++u) {
    quantise<T>(raw[u], c[u], s[u]);
    if constexpr (VALUES) {
      const int64_t i = first + u * MOE_WAVE + lane;
      if (i < pieces) moe::store_nt16(values + i, values_of<T>(c[u], s[u]));
    }
  }
  const int q = lane & 3;
  if constexpr (sizeof(T) == 2) {
    uint32_t o[4] = {};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t d[4] = {dpp<0x00>(c[u]), dpp<0x55>(c[u]), dpp<0xAA>(c[u]), dpp<0xFF>(c[u])};
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = q == u ? d[r] : o[r];
    }
    const uint32_t sq = q == 0 ? s[0] : q == 1 ? s[1] : q == 2 ? s[2] : s[3];
    const int64_t block = (first + q * MOE_WAVE + lane) >> 2;
    if (block < pieces >> 2) {
      moe::store_nt16(codes + block * 16, make_uint4(o[0], o[1], o[2], o[3]));
      scales[block] = static_cast<uint8_t>(sq);
    }
  } else {
    // even lanes keep chunks 0 and 1, odd lanes 2 and 3
    const bool odd = lane & 1;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t n0 = dpp<kXor1>(c[u]), n1 = dpp<kXor1>(c[u + 2]);
      const uint32_t d = odd ? n1 | c[u + 2] << 16 : c[u] | n0 << 16;
      const int64_t i = first + (odd ? u + 2 : u) * MOE_WAVE + (lane & ~1);
      if (i < pieces) reinterpret_cast<uint32_t*>(codes)[i >> 1] = d;
    }
    const uint32_t sq = q == 0 ? s[0] : q == 1 ? s[1] : q == 2 ? s[2] : s[3];
    const int64_t block = (first + q * MOE_WAVE + lane) >> 3;
    if ((lane & 4) == 0 && block < pieces >> 3) scales[block] = static_cast<uint8_t>(sq);
  }
}

template <typename T>
moe_status launch_quantize(const void* x, int64_t total, void* codes, void* scales, void* values, hipStream_t stream) {
  constexpr int per = 16 / sizeof(T), block = 4 * kChunks * MOE_WAVE;   // values of a piece, pieces of a workgroup
  constexpr int64_t most = kMaxLanes / 256 * block;
  const int64_t pieces = total / per;
  for (int64_t at = 0; at < pieces; at += most) {
    const int64_t n = pieces - at < most ? pieces - at : most;
    const int grid = static_cast<int>((n + block - 1) / block);
    const uint4* xs = static_cast<const uint4*>(x) + at;
    uint8_t* cs = static_cast<uint8_t*>(codes) + at * (per / 2);
    uint8_t* ss = static_cast<uint8_t*>(scales) + at * per / 32;
    if (values)
      quantize_kernel<T, true><<<grid, 256, 0, stream>>>(xs, n, cs, ss, static_cast<uint4*>(values) + at);
    else
      quantize_kernel<T, false><<<grid, 256, 0, stream>>>(xs, n, cs, ss, nullptr);
    MOE_LAUNCH_CHECK();
  }
  return MOE_OK;
}

// ---------------------------------------------------------------- dispatch

// One wave per (token, part of its row): lane k reads route k, a ballot gives the
// local routes, the part is read and quantised once and stored once per route.
// Pairs of lanes exchange codes so that the even lane stores both lanes' of the
// even chunk and the odd lane of the odd one.
constexpr int kRowWaves = 4;                     // of a workgroup (one: 16.4 us at prefill, four 14.7)

template <typename T, int PART>                  // PART chunks of a row
__global__ __launch_bounds__(kRowWaves * MOE_WAVE) void permute_mx4_kernel(const uint4* __restrict__ x, int tokens, int K,
                                                                          int H, const int32_t* __restrict__ slot_of,
                                                                          int64_t rows_cap, uint8_t* __restrict__ buf,
                                                                          uint8_t* __restrict__ scales, int parts) {
  constexpr int per = 16 / sizeof(T), lanes = 32 / per;                        // values of a piece, lanes of a block
  const int lane = moe::lane_id();
  const int item = blockIdx.x * kRowWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = item / parts;
  const int p = item - t * parts;
  if (t >= tokens) return;
  const int s_l = lane < K ? slot_of[static_cast<int64_t>(t) * K + lane] : -1;
  const uint64_t routes = __ballot(s_l >= 0 && s_l < rows_cap);
  if (!routes) return;
  const int pieces = H / per;
  const uint4* src = x + static_cast<int64_t>(t) * pieces;
  uint4 raw[PART];
#pragma unroll
  for (int u = 0; u < PART; ++u) {
    const int i = (p * PART + u) * MOE_WAVE + lane;
    raw[u] = i < pieces ? src[i] : make_uint4(0, 0, 0, 0);
  }
  uint32_t c[PART], s[PART];
#pragma unroll
  for (int u = 0; u < PART; ++u) quantise<T>(raw[u], c[u], s[u]);
  const bool odd = lane & 1;
  uint32_t lo[PART / 2], hi[PART / 2], sq[PART / 2];
#pragma unroll
  for (int u = 0; u < PART / 2; ++u) {
    const uint32_t c0 = c[2 * u], c1 = c[2 * u + 1], n0 = dpp<kXor1>(c0), n1 = dpp<kXor1>(c1);
    const uint32_t s0 = s[2 * u], s1 = s[2 * u + 1];
    sq[u] = odd ? s1 : s0;
    if constexpr (sizeof(T) == 2) lo[u] = odd ? n1 : c0, hi[u] = odd ? c1 : n0;
    else lo[u] = odd ? n1 | c1 << 16 : c0 | n0 << 16, hi[u] = 0;
  }
  for (uint64_t m = routes; m; m &= m - 1) {
    const int64_t q = __builtin_amdgcn_readlane(s_l, __builtin_ctzll(m));
#pragma unroll
    for (int u = 0; u < PART / 2; ++u) {
      const int at = (p * PART + 2 * u + (odd ? 1 : 0)) * MOE_WAVE + (lane & ~1);     // first piece of the two
      if (at < pieces) {
        if constexpr (sizeof(T) == 2) reinterpret_cast<uint2*>(buf + q * (H / 2))[at >> 1] = make_uint2(lo[u], hi[u]);
        else reinterpret_cast<uint32_t*>(buf + q * (H / 2))[at >> 1] = lo[u];
        if ((lane & (lanes - 2)) == 0) scales[q * (H / 32) + at / lanes] = static_cast<uint8_t>(sq[u]);
      }
    }
  }
}

template <typename T, int PART>
moe_status launch_parts(const void* x, int tokens, int K, int H, const int32_t* slot_of, int64_t rows_cap, void* buf,
                        void* buf_scales, hipStream_t stream) {
  const int pieces = H / (16 / sizeof(T)), parts = (pieces + PART * MOE_WAVE - 1) / (PART * MOE_WAVE);
  const int64_t most = kMaxLanes / MOE_WAVE / parts;                           // tokens of a launch
  for (int64_t t = 0; t < tokens; t += most) {
    const int n = static_cast<int>(tokens - t < most ? tokens - t : most);
    permute_mx4_kernel<T, PART><<<(n * parts + kRowWaves - 1) / kRowWaves, kRowWaves * MOE_WAVE, 0, stream>>>(
        static_cast<const uint4*>(x) + t * pieces, n, K, H, slot_of + t * K, rows_cap, static_cast<uint8_t*>(buf),
        static_cast<uint8_t*>(buf_scales), parts);
    MOE_LAUNCH_CHECK();
  }
  return MOE_OK;
}

// Four chunks a wave where rows fill two such parts and the parts fill the chip's 8192 places for waves: more loads in flight.
// Two against four, us: 8192 x 7168 bf16 14.7 and 13.2, fp32 27.2 and 24.5; 128 x 7168 2.3 and 2.7; 1000 x 1408 2.4 and 2.7;
// 16384 x 512 5.1 and 6.6.
template <typename T>
moe_status launch_permute(const void* x, int tokens, int K, int H, const int32_t* slot_of, int64_t rows_cap, void* buf,
                          void* buf_scales, hipStream_t stream) {
  const int64_t pieces = H / (16 / sizeof(T)), parts = (pieces + 4 * MOE_WAVE - 1) / (4 * MOE_WAVE);
  return (pieces >= 8 * MOE_WAVE && tokens * parts >= 8192 ? launch_parts<T, 4> : launch_parts<T, 2>)(
      x, tokens, K, H, slot_of, rows_cap, buf, buf_scales, stream);
}

// ---------------------------------------------------------------- packing

// One thread moves one 16-byte piece.
__global__ __launch_bounds__(256) void pack_mx4_codes_kernel(const uint4* __restrict__ codes, int64_t pieces, int steps,
                                                             uint4* __restrict__ out) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < pieces; i += gridDim.x * 256ll) {
    const int l = static_cast<int>(i & 63);
    const int64_t blk = i >> 6;
    const int64_t nt = blk / steps;                // (expert, 16-row tile)
    const int ks = static_cast<int>(blk - nt * steps);
    out[i] = codes[((nt * 16 + (l & 15)) * steps + ks) * 4 + (l >> 4)];
  }
}

// One thread makes the bytes of one piece place l in up to four steps.
__global__ __launch_bounds__(256) void pack_mx4_scales_kernel(const uint8_t* __restrict__ scales, int64_t count,
                                                              int steps, uint8_t* __restrict__ out) {
  const int groups = (steps + 3) / 4;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < count; i += gridDim.x * 256ll) {
    const int l = static_cast<int>(i & 63);
    const int64_t blk = i >> 6;
    const int64_t nt = blk / groups;
    const int g = static_cast<int>(blk - nt * groups);
    const int n = steps - 4 * g < 4 ? steps - 4 * g : 4;
    const uint8_t* src = scales + ((nt * 16 + (l & 15)) * steps + 4 * g) * 4 + (l >> 4);
    uint8_t* dst = out + (nt * steps + 4 * g) * 64 + l * n;
    for (int j = 0; j < n; ++j) dst[j] = src[4 * j];
  }
}

}  // namespace

extern "C" moe_status moe_quantize_mx4(const void* x, moe_dtype x_dt, int64_t rows, int K, void* codes, void* scales,
                                       void* values, hipStream_t stream) {
  MOE_CHECK(rows >= 0 && K > 0 && moe_host::valid_dtype(x_dt), MOE_ERR_INVALID_ARG);
  MOE_CHECK(K % 32 == 0 && real_dtype(x_dt) && rows <= (1ll << 40) / K, MOE_ERR_UNSUPPORTED);
  if (rows == 0) return MOE_OK;
  MOE_CHECK(x && codes && scales, MOE_ERR_INVALID_ARG);
  MOE_CHECK(aligned(x, 16) && aligned(codes, 16) && aligned(values, 16), MOE_ERR_INVALID_ARG);
  return x_dt == MOE_F32 ? launch_quantize<float>(x, rows * K, codes, scales, values, stream)
                         : launch_quantize<uint16_t>(x, rows * K, codes, scales, values, stream);
}

extern "C" moe_status moe_permute_mx4(const void* x, moe_dtype x_dt, int T, int K, int H, const int32_t* slot_of,
                                      int64_t rows_cap, void* buf, void* buf_scales, hipStream_t stream) {
  MOE_CHECK(T >= 0 && K > 0 && H > 0 && rows_cap >= 0 && moe_host::valid_dtype(x_dt), MOE_ERR_INVALID_ARG);
  MOE_CHECK(H % 32 == 0 && H <= 1 << 25 && K <= 64 && real_dtype(x_dt), MOE_ERR_UNSUPPORTED);
  MOE_CHECK(static_cast<int64_t>(T) * ((H + 1023) / 1024) <= 0x7fffffff, MOE_ERR_UNSUPPORTED);
  if (T == 0 || rows_cap == 0) return MOE_OK;
  MOE_CHECK(x && slot_of && buf && buf_scales, MOE_ERR_INVALID_ARG);
  MOE_CHECK(aligned(x, 16) && aligned(buf, 16), MOE_ERR_INVALID_ARG);
  return x_dt == MOE_F32 ? launch_permute<float>(x, T, K, H, slot_of, rows_cap, buf, buf_scales, stream)
                         : launch_permute<uint16_t>(x, T, K, H, slot_of, rows_cap, buf, buf_scales, stream);
}

extern "C" moe_status moe_pack_mx4(const void* codes, const void* scales, int L, int N, int K, void* codes_packed,
                                   void* scales_packed, hipStream_t stream) {
  MOE_CHECK(L > 0 && N > 0 && K > 0, MOE_ERR_INVALID_ARG);
  MOE_CHECK(L <= 1024 && N % 16 == 0 && K % 128 == 0 && K <= 1 << 24 && static_cast<int64_t>(N) * K <= 1ll << 31 &&
                static_cast<int64_t>(L) * N * K < 1ll << 39, MOE_ERR_UNSUPPORTED);
  MOE_CHECK(codes && scales && codes_packed && scales_packed && codes != codes_packed && scales != scales_packed,
            MOE_ERR_INVALID_ARG);
  MOE_CHECK(aligned(codes, 16) && aligned(codes_packed, 16) && aligned(scales, 4) && aligned(scales_packed, 4),
            MOE_ERR_INVALID_ARG);
  const int steps = K / 128;
  const int64_t pieces = static_cast<int64_t>(L) * N * (K / 32);
  const int64_t count = static_cast<int64_t>(L) * N / 16 * ((steps + 3) / 4) * 64;
  auto grid = [](int64_t n) { return static_cast<int>((n + 255) / 256 < 16384 ? (n + 255) / 256 : 16384); };
  pack_mx4_codes_kernel<<<grid(pieces), 256, 0, stream>>>(static_cast<const uint4*>(codes), pieces, steps,
                                                          static_cast<uint4*>(codes_packed));
  MOE_LAUNCH_CHECK();
  pack_mx4_scales_kernel<<<grid(count), 256, 0, stream>>>(static_cast<const uint8_t*>(scales), count, steps,
                                                          static_cast<uint8_t*>(scales_packed));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}
