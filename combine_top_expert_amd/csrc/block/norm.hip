// moe_add_rms_norm and its backward.
//
// Forward: h = x + residual (rounded to the storage type), y = h r w with
// r = 1 / sqrt(mean h^2 + eps), written as bf16/fp32 rows and/or block FP8.
// Backward: dx = dh + r (w dy - n mean(w dy n)), n = h r; d_w = sum_t dy n.
//
// A group of WAVES wavefronts owns a row and holds it in registers as chunks
// of 8 neighbouring columns (chunk c of lane i: 8 (64 WAVES v + i)), so a row
// is read once and every access is 16 bytes per lane.  Sums run in fp32: per
// lane, a DPP wave sum, then the waves' sums through LDS in wave order.  A
// group of 128 columns is 16 neighbouring lanes, whose amax is an in-row DPP
// maximum.

#include "block_common.h"
#include "router_common.h"

namespace {

using namespace moe_block;

constexpr int kMaxH = 16384;

// Sum over the WAVES waves of the block; every thread gets it.  `red` has
// WAVES entries; the leading barrier covers reads of an earlier call's values.
template <int WAVES> __device__ __forceinline__ float block_sum(float v, float* red) {
  v = moe_router::wave_sum_f32(v);
  if constexpr (WAVES == 1) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) s += red[i];
  return s;
}

template <typename T, typename TW, int WAVES, int VPL>
__global__ __launch_bounds__(WAVES * 64) void add_rms_norm_kernel(const T* x, const T* residual,
                                                                 const TW* __restrict__ weight, float eps, int H,
                                                                 T* h_out, T* y, uint8_t* __restrict__ y8,
                                                                 float* __restrict__ scales) {
  __shared__ float red[WAVES];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * H;
  float h[VPL][8];
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = (v * WAVES * 64 + threadIdx.x) * 8;
    if (c < H) {
      load8(x + base + c, h[v]);
      if (residual) {
        float r[8];
        load8(residual + base + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = as_stored<T>(h[v][i] + r[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
    }
  }
  const float r = 1.0f / sqrtf(block_sum<WAVES>(ss, red) / static_cast<float>(H) + eps);
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = (v * WAVES * 64 + threadIdx.x) * 8;
    if (c < H) {
      if (h_out) store8(h_out + base + c, h[v]);
      float w[8];
      load8(weight + c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * r * w[i];
      if (y) store8(y + base + c, h[v]);
      if (y8) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(h[v][i]));
        amax = moe::fp8_group_amax_clamp(moe_router::row_max_f32(amax));
        const float inv = moe::fp8_group_inv(amax);
        *reinterpret_cast<uint2*>(y8 + base + c) =
            make_uint2(moe::f32x4_to_e4m3(h[v][0] * inv, h[v][1] * inv, h[v][2] * inv, h[v][3] * inv),
                       moe::f32x4_to_e4m3(h[v][4] * inv, h[v][5] * inv, h[v][6] * inv, h[v][7] * inv));
        if ((threadIdx.x & 15) == 0) scales[(base + c) >> 7] = moe::fp8_group_scale(amax);
      }
    }
  }
}

// Rows of the backward that one block walks: block b takes rows b, b + G, ...
// and keeps its share of d_w in registers, written once as row b of the
// workspace [G, H].
constexpr int kBwBlocks = 512;
inline int bw_blocks(int T) { return T < kBwBlocks ? T : kBwBlocks; }

template <typename T, typename TW, int WAVES, int VPL>
__global__ __launch_bounds__(WAVES * 64) void add_rms_norm_bw_kernel(const T* dy, const T* h, const T* dh,
                                                                    const TW* __restrict__ weight, float eps,
                                                                    int rows, int H, T* dx,
                                                                    float* __restrict__ part) {
  __shared__ float red[2][WAVES];
  float dw[VPL][8] = {};
  for (int t = blockIdx.x; t < rows; t += gridDim.x) {
    const int64_t base = static_cast<int64_t>(t) * H;
    float hv[VPL][8], g[VPL][8];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = (v * WAVES * 64 + threadIdx.x) * 8;
      if (c < H) {
        float w[8];
        load8(h + base + c, hv[v]);
        load8(dy + base + c, g[v]);
        load8(weight + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(hv[v][i], hv[v][i], ss);
          dot = fmaf(hv[v][i], g[v][i] * w[i], dot);
        }
      }
    }
    const float r = 1.0f / sqrtf(block_sum<WAVES>(ss, red[0]) / static_cast<float>(H) + eps);
    const float k = block_sum<WAVES>(dot, red[1]) * r / static_cast<float>(H);   // mean(w dy n)
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = (v * WAVES * 64 + threadIdx.x) * 8;
      if (c < H) {
        float w[8], o[8];
        load8(weight + c, w);
        if (dh) load8(dh + base + c, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = hv[v][i] * r;
          dw[v][i] = fmaf(g[v][i], n, dw[v][i]);
          const float d = r * (g[v][i] * w[i] - n * k);
          o[i] = dh ? o[i] + d : d;
        }
        store8(dx + base + c, o);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = (v * WAVES * 64 + threadIdx.x) * 8;
    if (c < H) store8(part + static_cast<int64_t>(blockIdx.x) * H + c, dw[v]);
  }
}

// d_w[c] = sum_b part[b, c]: a block takes 64 columns, its 16 waves every 16th
// row; the waves' sums meet in LDS and are added in wave order.
constexpr int kRedWaves = 16;
__global__ __launch_bounds__(kRedWaves * 64) void reduce_dw_kernel(const float* __restrict__ part, int nblk, int H,
                                                                  float* __restrict__ dw) {
  __shared__ float red[kRedWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < H)
    for (int b = wave; b < nblk; b += kRedWaves) s += part[static_cast<int64_t>(b) * H + c];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < H) {
    for (int i = 1; i < kRedWaves; ++i) s += red[i][lane];
    dw[c] = s;
  }
}

struct FwArgs {
  const void *x, *residual, *weight;
  float eps;
  int T, H;
  void *h_out, *y;
  uint8_t* y8;
  float* scales;
  hipStream_t stream;
};

template <typename T, typename TW, int WAVES, int VPL> void fw_launch(const FwArgs& a) {
  add_rms_norm_kernel<T, TW, WAVES, VPL><<<a.T, WAVES * 64, 0, a.stream>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.residual), static_cast<const TW*>(a.weight), a.eps, a.H,
      static_cast<T*>(a.h_out), static_cast<T*>(a.y), a.y8, a.scales);
}

// WAVES so that a row is at most two chunks per lane.
template <typename T, typename TW> void fw_pick(const FwArgs& a) {
  const int chunks = a.H / 8;
  if (chunks <= 64) fw_launch<T, TW, 1, 1>(a);
  else if (chunks <= 128) fw_launch<T, TW, 2, 1>(a);
  else if (chunks <= 256) fw_launch<T, TW, 4, 1>(a);
  else if (chunks <= 512) fw_launch<T, TW, 4, 2>(a);
  else if (chunks <= 1024) fw_launch<T, TW, 8, 2>(a);
  else fw_launch<T, TW, 16, 2>(a);
}

struct BwArgs {
  const void *dy, *h, *dh, *weight;
  float eps;
  int T, H;
  void* dx;
  float* part;
  int nblk;
  hipStream_t stream;
};

template <typename T, typename TW, int WAVES, int VPL> void bw_launch(const BwArgs& a) {
  add_rms_norm_bw_kernel<T, TW, WAVES, VPL><<<a.nblk, WAVES * 64, 0, a.stream>>>(
      static_cast<const T*>(a.dy), static_cast<const T*>(a.h), static_cast<const T*>(a.dh),
      static_cast<const TW*>(a.weight), a.eps, a.T, a.H, static_cast<T*>(a.dx), a.part);
}

template <typename T, typename TW> void bw_pick(const BwArgs& a) {
  const int chunks = a.H / 8;
  if (chunks <= 64) bw_launch<T, TW, 1, 1>(a);
  else if (chunks <= 128) bw_launch<T, TW, 2, 1>(a);
  else if (chunks <= 256) bw_launch<T, TW, 4, 1>(a);
  else if (chunks <= 512) bw_launch<T, TW, 4, 2>(a);
  else if (chunks <= 1024) bw_launch<T, TW, 8, 2>(a);
  else bw_launch<T, TW, 16, 2>(a);
}

inline bool norm_sizes(int T, int H) { return T >= 0 && H > 0; }
inline bool good_eps(float eps) { return eps >= 0.f && eps < INFINITY; }

}  // namespace

extern "C" moe_status moe_add_rms_norm(const void* x, const void* residual, moe_dtype x_dt, const void* weight,
                                       moe_dtype w_dt, float eps, int T, int H, void* h_out, void* y, void* y8,
                                       float* y8_scales, hipStream_t stream) {
  MOE_CHECK(norm_sizes(T, H) && good_eps(eps), MOE_ERR_INVALID_ARG);
  MOE_CHECK(moe_host::valid_dtype(x_dt) && moe_host::valid_dtype(w_dt), MOE_ERR_INVALID_ARG);
  MOE_CHECK(real_dtype(x_dt) && real_dtype(w_dt), MOE_ERR_UNSUPPORTED);
  MOE_CHECK(H % 8 == 0 && H <= kMaxH, MOE_ERR_UNSUPPORTED);
  MOE_CHECK(h_out || y || y8 || T == 0, MOE_ERR_INVALID_ARG);
  MOE_CHECK(!y8 == !y8_scales, MOE_ERR_INVALID_ARG);
  MOE_CHECK(!y8 || H % 128 == 0, MOE_ERR_UNSUPPORTED);
  if (T == 0) return MOE_OK;
  MOE_CHECK(x && weight && (!y || y != h_out), MOE_ERR_INVALID_ARG);
  MOE_CHECK(aligned16(x) && aligned16(residual) && aligned16(weight) && aligned16(h_out) && aligned16(y) && aligned16(y8),
            MOE_ERR_INVALID_ARG);
  const FwArgs a{x, residual, weight, eps, T, H, h_out, y, static_cast<uint8_t*>(y8), y8_scales, stream};
  if (x_dt == MOE_BF16) {
    if (w_dt == MOE_BF16) fw_pick<uint16_t, uint16_t>(a);
    else fw_pick<uint16_t, float>(a);
  } else {
    if (w_dt == MOE_BF16) fw_pick<float, uint16_t>(a);
    else fw_pick<float, float>(a);
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

extern "C" size_t moe_add_rms_norm_backward_workspace_bytes(int T, int H) {
  if (!norm_sizes(T, H) || H % 8 != 0 || H > kMaxH) return 0;
  return static_cast<size_t>(bw_blocks(T)) * H * sizeof(float);
}

extern "C" moe_status moe_add_rms_norm_backward(const void* dy, const void* h, const void* dh, moe_dtype dt,
                                                const void* weight, moe_dtype w_dt, float eps, int T, int H,
                                                void* dx, float* d_weight, void* workspace, size_t workspace_bytes,
                                                hipStream_t stream) {
  MOE_CHECK(norm_sizes(T, H) && good_eps(eps), MOE_ERR_INVALID_ARG);
  MOE_CHECK(moe_host::valid_dtype(dt) && moe_host::valid_dtype(w_dt), MOE_ERR_INVALID_ARG);
  MOE_CHECK(real_dtype(dt) && real_dtype(w_dt), MOE_ERR_UNSUPPORTED);
  MOE_CHECK(H % 8 == 0 && H <= kMaxH, MOE_ERR_UNSUPPORTED);
  MOE_CHECK(d_weight && aligned16(d_weight), MOE_ERR_INVALID_ARG);
  const size_t need = moe_add_rms_norm_backward_workspace_bytes(T, H);
  if (T > 0) {
    MOE_CHECK(dy && h && weight && dx && workspace, MOE_ERR_INVALID_ARG);
    MOE_CHECK(aligned16(dy) && aligned16(h) && aligned16(dh) && aligned16(weight) && aligned16(dx) && aligned16(workspace),
              MOE_ERR_INVALID_ARG);
    MOE_CHECK(workspace_bytes >= need, MOE_ERR_WORKSPACE);
    const BwArgs a{dy, h, dh, weight, eps, T, H, dx, static_cast<float*>(workspace), bw_blocks(T), stream};
    if (dt == MOE_BF16) {
      if (w_dt == MOE_BF16) bw_pick<uint16_t, uint16_t>(a);
      else bw_pick<uint16_t, float>(a);
    } else {
      if (w_dt == MOE_BF16) bw_pick<float, uint16_t>(a);
      else bw_pick<float, float>(a);
    }
    MOE_LAUNCH_CHECK();
  }
  reduce_dw_kernel<<<(H + 63) / 64, kRedWaves * 64, 0, stream>>>(static_cast<const float*>(workspace),
                                                                 T > 0 ? bw_blocks(T) : 0, H, d_weight);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}
