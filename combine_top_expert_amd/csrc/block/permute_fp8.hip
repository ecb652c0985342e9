// moe_permute_fp8: block-FP8 token rows and their scales into the expert-major
// buffer, copied bit for bit.
//
// One wave per (token, 2 KB part of its row), one wave per workgroup: lane k
// reads route k, a ballot gives the local routes, the part is read once (1 KB
// per load) and stored once per route.  A 2 KB part has 16 scales, which 16
// lanes carry along.
//
// Bound by memory: 8192 tokens of 7168 codes, 8192 routes to 32 of 256 experts
// (100 MB read and written) take 9.4 us where the 256 MB cache holds them; a
// decode step's 128 tokens take 2.3 us, a launch.

#include "block_common.h"

namespace {

constexpr int kLoads = 2;
constexpr int kChunks = kLoads * MOE_WAVE;      // 16-byte chunks of a part

__global__ __launch_bounds__(MOE_WAVE) void permute_fp8_kernel(const uint8_t* __restrict__ x,
                                                              const float* __restrict__ xs, int T, int K, int H,
                                                              const int32_t* __restrict__ slot_of, int64_t rows_cap,
                                                              uint8_t* __restrict__ buf, float* __restrict__ scales,
                                                              int parts) {
  const int lane = moe::lane_id();
  const int t = blockIdx.x / parts;
  const int p = blockIdx.x - t * parts;
  const int s_l = lane < K ? slot_of[static_cast<int64_t>(t) * K + lane] : -1;
  const uint64_t routes = __ballot(s_l >= 0 && s_l < rows_cap);
  if (!routes) return;
  const int nchunk = H / 16, groups = H / 128;
  const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(t) * H);
  uint4 raw[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int c = p * kChunks + u * MOE_WAVE + lane;
    raw[u] = c < nchunk ? src[c] : make_uint4(0, 0, 0, 0);
  }
  const int g = p * (kChunks / 8) + lane;
  const bool has_scale = lane < kChunks / 8 && g < groups;
  const float sc = has_scale ? xs[static_cast<int64_t>(t) * groups + g] : 0.f;
  for (uint64_t m = routes; m; m &= m - 1) {
    const int64_t s = __builtin_amdgcn_readlane(s_l, __builtin_ctzll(m));
    uint4* dst = reinterpret_cast<uint4*>(buf + s * H);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int c = p * kChunks + u * MOE_WAVE + lane;
      if (c < nchunk) moe::store_nt16(dst + c, raw[u]);
    }
    if (has_scale) scales[s * groups + g] = sc;
  }
}

}  // namespace

extern "C" moe_status moe_permute_fp8(const void* x8, const float* x8_scales, int T, int K, int H,
                                      const int32_t* slot_of, int64_t rows_cap, void* buf, float* buf_scales,
                                      hipStream_t stream) {
  MOE_CHECK(T >= 0 && K > 0 && H > 0 && rows_cap >= 0, MOE_ERR_INVALID_ARG);
  MOE_CHECK(H % 128 == 0 && K <= 64, MOE_ERR_UNSUPPORTED);
  if (T == 0 || rows_cap == 0) return MOE_OK;
  MOE_CHECK(x8 && x8_scales && slot_of && buf && buf_scales, MOE_ERR_INVALID_ARG);
  MOE_CHECK(moe_block::aligned16(x8) && moe_block::aligned16(buf), MOE_ERR_INVALID_ARG);
  const int parts = (H / 16 + kChunks - 1) / kChunks;
  const int64_t grid = static_cast<int64_t>(T) * parts;
  MOE_CHECK(grid <= 0x7fffffff && parts <= 1 << 14, MOE_ERR_UNSUPPORTED);
  return moe_block::in_slices(T, static_cast<int64_t>(parts) * MOE_WAVE, [&](int64_t t, int rows) {
    permute_fp8_kernel<<<rows * parts, MOE_WAVE, 0, stream>>>(
        static_cast<const uint8_t*>(x8) + t * H, x8_scales + t * (H / 128), rows, K, H, slot_of + t * K, rows_cap,
        static_cast<uint8_t*>(buf), buf_scales, parts);
  });
}
