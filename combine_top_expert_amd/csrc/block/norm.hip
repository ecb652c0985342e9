// moe_add_rms_norm and its backward.
//
// Forward: h = x + residual (rounded to the storage type), y = h r w with
// r = 1 / sqrt(mean h^2 + eps), written as bf16/fp32 rows and/or block FP8.
// Backward: dx = dh + r (w dy - n mean(w dy n)), n = h r; d_w = sum_t dy n.
//
// A block owns a row and holds it in registers as chunks of 8 neighbouring
// columns (chunk v of thread i: columns 8 (threads v + i)), so a row is read
// once and every access is 16 bytes per lane.  Sums run in fp32: per
// lane, a DPP wave sum, then the waves' sums through LDS in wave order.  A
// group of 128 columns is 16 neighbouring lanes, whose amax is an in-row DPP
// maximum.  It keeps a NaN: a lane's eight magnitudes meet in the maximum that
// does, the lanes' in one of their bits (as integers they have the values' order,
// with NaN above infinity).  The conversion to e4m3 clamps, which makes a NaN
// -448, so groups whose amax is no finite number are looked at once more.
//
// Bound by memory.  Forward, 8192 x 7168 bf16 with residual to h and FP8 (413
// MB): 69.6 to 72 us, 5.9 TB/s; backward, 16384 x 4096 bf16 with dh (537 MB): 91.5
// to 95 us and 4.2 for the reduction of d_w, 5.6 TB/s.

#include "block_common.h"
#include "router_common.h"

namespace {

using namespace moe_block;

constexpr int kMaxH = 16384;
constexpr int kMaxWaves = 16;

// Sums over the block's waves of two values; every thread gets them, added in
// wave order.  `red` must not be the array of the call before (one barrier
// orders the writes before the reads, and only that).
__device__ __forceinline__ float2 block_sum(float u, float v, int waves, float2* red) {
  u = moe_router::wave_sum_f32(u);
  v = moe_router::wave_sum_f32(v);
  if (waves == 1) return make_float2(u, v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = make_float2(u, v);
  __syncthreads();
  float2 s = red[0];
  for (int i = 1; i < waves; ++i) {
    s.x += red[i].x;
    s.y += red[i].y;
  }
  return s;
}

// 16 bytes, with NT past the caches' retention: from 32 MB of rows on, what a
// call reads and writes does not stay in the 32 MB of L2 in any case
// (measured below).
template <bool NT> __device__ __forceinline__ uint4 get16(const void* p) {
  return NT ? moe::load_nt16(p) : *reinterpret_cast<const uint4*>(p);
}
template <bool NT> __device__ __forceinline__ void put16(void* p, const uint4& v) {
  if (NT) moe::store_nt16(p, v);
  else *reinterpret_cast<uint4*>(p) = v;
}

// Eight neighbouring elements as loaded.
template <typename T> struct Chunk;
template <> struct Chunk<float> {
  uint4 a, b;
  template <bool NT> __device__ __forceinline__ void load(const float* p) {
    a = get16<NT>(p);
    b = get16<NT>(p + 4);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
  }
};
template <> struct Chunk<uint16_t> {
  uint4 a;
  template <bool NT> __device__ __forceinline__ void load(const uint16_t* p) { a = get16<NT>(p); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <bool NT> __device__ __forceinline__ void put(float* p, const float* f) {
  put16<NT>(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
  put16<NT>(p + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
}
template <bool NT> __device__ __forceinline__ void put(uint16_t* p, const float* f) {
  put16<NT>(p, make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
}

// One row per block of `waves` wavefronts; lane i of the block holds the chunks
// i, i + 64 waves, ... (VPL of them).
template <typename T, typename TW, int VPL, bool NT>
__global__ __launch_bounds__(kMaxWaves * 64) void add_rms_norm_kernel(const T* x, const T* residual,
                                                                     const TW* __restrict__ weight, float eps, int H,
                                                                     T* h_out, T* y, uint8_t* __restrict__ y8,
                                                                     float* __restrict__ scales) {
  __shared__ float2 red[kMaxWaves];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * H;
  const int threads = blockDim.x;
  Chunk<T> cx[VPL], cr[VPL];
  Chunk<TW> cw[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = (v * threads + threadIdx.x) * 8;
    if (c < H) {
      cx[v].template load<NT>(x + base + c);
      if (residual) cr[v].template load<NT>(residual + base + c);
      cw[v].template load<false>(weight + c);
    }
  }
  float h[VPL][8];
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = (v * threads + threadIdx.x) * 8;
    if (c < H) {
      cx[v].get(h[v]);
      if (residual) {
        float r[8];
        cr[v].get(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = as_stored<T>(h[v][i] + r[i]);
        if (h_out) put<NT>(h_out + base + c, h[v]);
      } else if (h_out) {
        put<NT>(h_out + base + c, h[v]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
    }
  }
  if (!y && !y8) return;
  const float r = 1.0f / sqrtf(block_sum(ss, 0.f, threads >> 6, red).x / static_cast<float>(H) + eps);
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = (v * threads + threadIdx.x) * 8;
    if (c < H) {
      float w[8];
      cw[v].get(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * r * w[i];
      if (y) put<NT>(y + base + c, h[v]);
      if (y8) {
        float top = moe::fp8_group_amax_clamp(0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = __builtin_elementwise_maximum(top, fabsf(h[v][i]));
        const float amax = __uint_as_float(moe_router::row_max_u32(__float_as_uint(top)));
        const float inv = moe::fp8_group_inv(amax);
        uint2 code = make_uint2(moe::f32x4_to_e4m3(h[v][0] * inv, h[v][1] * inv, h[v][2] * inv, h[v][3] * inv),
                                moe::f32x4_to_e4m3(h[v][4] * inv, h[v][5] * inv, h[v][6] * inv, h[v][7] * inv));
        if (!(amax < INFINITY)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float q = h[v][i] * inv;
            if (q != q) (i < 4 ? code.x : code.y) |= 0x7fu << (8 * (i & 3));
          }
        }
        *reinterpret_cast<uint2*>(y8 + base + c) = code;
        if ((threadIdx.x & 15) == 0) scales[(base + c) >> 7] = moe::fp8_group_scale(amax);
      }
    }
  }
}

// Rows of the backward that one block walks: block b takes rows b, b + G, ...
// and keeps its share of d_w in registers, written once as row b of the
// workspace [G, H].  The next row's loads are issued before this row's sums.
// 16384 x 4096 bf16 in us, 512 / 1024 blocks: 95 / 91 with the reduction's 5;
// 1001 x 1408 fp32, 512 / 768 / 1024: 10 / 11 / 12.  Narrow rows have few waves
// a block and get more blocks, with 32 rows each at least (65536 x 512 bf16,
// 1024 / 2048 / 4096 blocks: 66 / 57 / 59; 32768 x 1408, 1024 / 2048: 68 / 82).
// Wider and fp32 rows, reduction included, 256 / 512 / 1024 / 2048 blocks: bf16
// 1024 x 7168 21.3 / 21.9 / 26.8 / 26.8; 2048 x 7168 34.7 / 32.4 / 37.9 / 46.8; 8192 x
// 7168 110 / 88 / 91 / 102; 8192 x 5120 102 / 64 / 85 / 82 (there the rule's 1024 are
// not the best); 2048 x 16384 56 / 65 / 84 / 110; fp32 1024 x 7168 31 / 36 / 41 / 41;
// 8192 x 7168 194 / 198 / 206 / 220; 8192 x 4096 123 / 103 / 107 / 115; 16384 x 1408 121 /
// 88 / 76 / 85.
inline int bw_blocks(int T, int H) {
  const int waves = (H / 8 + 63) / 64;
  const int base = T >= 8192 ? 1024 : 512;
  const int narrow = 4096 / waves < T / 32 ? 4096 / waves : T / 32;
  const int most = base > narrow ? base : narrow;
  return T < most ? T : most;
}

template <typename T, typename TW, int VPL, bool NT>
__global__ __launch_bounds__(kMaxWaves * 64) void add_rms_norm_bw_kernel(const T* dy, const T* h, const T* dh,
                                                                        const TW* __restrict__ weight, float eps,
                                                                        int rows, int H, T* dx,
                                                                        float* __restrict__ part) {
  // (fp32 rows of two chunks a lane leave no registers for it)
  constexpr bool kAhead = !(sizeof(T) == 4 && VPL > 1);
  __shared__ float2 red[2][kMaxWaves];
  const int threads = blockDim.x;
  float dw[VPL][8] = {};
  Chunk<TW> w[VPL];
  struct Row {
    Chunk<T> h, dy, dh;
  } cur[VPL], next[VPL];
  auto fetch = [&](Row (&to)[VPL], int t) {
    const int64_t base = static_cast<int64_t>(t) * H;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = (v * threads + threadIdx.x) * 8;
      if (c < H) {
        to[v].h.template load<NT>(h + base + c);
        to[v].dy.template load<NT>(dy + base + c);
        if (dh) to[v].dh.template load<NT>(dh + base + c);
      }
    }
  };
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = (v * threads + threadIdx.x) * 8;
    if (c < H) w[v].template load<false>(weight + c);
  }
  fetch(cur, blockIdx.x);
  int parity = 0;
  for (int t = blockIdx.x; t < rows; t += gridDim.x) {
    if (kAhead && t + static_cast<int>(gridDim.x) < rows) fetch(next, t + gridDim.x);
    if (!kAhead && t != static_cast<int>(blockIdx.x)) fetch(cur, t);
    const int64_t base = static_cast<int64_t>(t) * H;
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = (v * threads + threadIdx.x) * 8;
      if (c < H) {
        float hv[8], g[8], wv[8];
        cur[v].h.get(hv);
        cur[v].dy.get(g);
        w[v].get(wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(hv[i], hv[i], ss);
          dot = fmaf(hv[i], g[i] * wv[i], dot);
        }
      }
    }
    const float2 s = block_sum(ss, dot, threads >> 6, red[parity]);
    parity ^= 1;
    const float r = 1.0f / sqrtf(s.x / static_cast<float>(H) + eps);
    const float k = s.y * r / static_cast<float>(H);   // mean(w dy n)
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = (v * threads + threadIdx.x) * 8;
      if (c < H) {
        float hv[8], g[8], wv[8], o[8];
        cur[v].h.get(hv);
        cur[v].dy.get(g);
        w[v].get(wv);
        if (dh) cur[v].dh.get(o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = hv[i] * r;
          dw[v][i] = fmaf(g[i], n, dw[v][i]);
          const float d = r * (g[i] * wv[i] - n * k);
          o[i] = dh ? o[i] + d : d;
        }
        put<NT>(dx + base + c, o);
      }
      if constexpr (kAhead) cur[v] = next[v];
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = (v * threads + threadIdx.x) * 8;
    if (c < H) put<false>(part + static_cast<int64_t>(blockIdx.x) * H + c, dw[v]);
  }
}

// d_w[c] = sum_b part[b, c]: a block takes 32 columns; 8 lanes of four columns
// side by side, ROWS of those take every ROWS-th row, and their sums are added
// in order from LDS.
constexpr int kRedCols = 32;
template <int ROWS>
__global__ __launch_bounds__(ROWS * 8) void reduce_dw_kernel(const float* __restrict__ part, int nblk, int H,
                                                             float* __restrict__ dw) {
  __shared__ float4 red[ROWS][kRedCols / 4];
  const int q = threadIdx.x % (kRedCols / 4), r = threadIdx.x / (kRedCols / 4);
  const int c = blockIdx.x * kRedCols + q * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < H)
#pragma unroll 8
    for (int b = r; b < nblk; b += ROWS) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(b) * H + c);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  red[r][q] = s;
  __syncthreads();
  if (threadIdx.x < kRedCols && blockIdx.x * kRedCols + static_cast<int>(threadIdx.x) < H) {
    const float* col = reinterpret_cast<const float*>(red) + threadIdx.x;
    float t = 0.f;
#pragma unroll 16
    for (int i = 0; i < ROWS; ++i) t += col[i * kRedCols];
    dw[blockIdx.x * kRedCols + threadIdx.x] = t;
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

// Rows of this many bytes in all go past the caches.
constexpr int64_t kStreamBytes = 32ll << 20;

template <typename T, typename TW, int VPL, bool NT> void fw_launch(const FwArgs& a) {
  const int waves = (a.H / 8 + 64 * VPL - 1) / (64 * VPL);
  add_rms_norm_kernel<T, TW, VPL, NT><<<a.T, waves * 64, 0, a.stream>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.residual), static_cast<const TW*>(a.weight), a.eps, a.H,
      static_cast<T*>(a.h_out), static_cast<T*>(a.y), a.y8, a.scales);
}

template <typename T, typename TW> void fw_pick(const FwArgs& a) {
  const bool nt = static_cast<int64_t>(a.T) * a.H * static_cast<int64_t>(sizeof(T)) >= kStreamBytes;
  // Below 32 MB: a row on as many waves as it has chunks for.  Past it: up to four
  // chunks a lane, so that a compute unit holds more rows at once (8192 x 7168
  // bf16 with residual to h and FP8, us: one chunk a lane 87, two 73.6, three
  // 73.3, four 71.1 = 5.8 TB/s, seven 75; two with plain loads and stores 79,
  // non-temporal loads only 79, stores only 76; codes stored past the
  // caches too 73.0).
  // With y as well, us for one / two / four: bf16, below 128 x 7168 5.1 / 5.7 / 7.7, 1024
  // x 7168 16.8 / 16.8 / 17.8, 2048 x 7168 29.0 / 30.4 / 33.0, 8192 x 1408 22.3 / 24.9 /
  // 26.1, past 4096 x 4096 27.9 / 28.2 / 31.6, 8192 x 7168 92 / 85 / 88; fp32, below 512 x
  // 7168 15.0 / 15.5 / 14.4, 1024 x 7168 26.3 / 27.4 / 27.5, past 4096 x 7168 96 / 103 /
  // 100, 8192 x 4096 107 / 111 / 116 (there one would be 4 % faster than the rule).
  const int chunks = a.H / 8;
  if (!nt) {
    if (chunks <= 64 * kMaxWaves) fw_launch<T, TW, 1, false>(a);
    else fw_launch<T, TW, 2, false>(a);
  } else {
    if (chunks <= 256) fw_launch<T, TW, 1, true>(a);
    else if (chunks <= 512) fw_launch<T, TW, 2, true>(a);
    else fw_launch<T, TW, 4, true>(a);
  }
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

template <typename T, typename TW, int VPL, bool NT> void bw_launch(const BwArgs& a) {
  const int waves = (a.H / 8 + 64 * VPL - 1) / (64 * VPL);
  add_rms_norm_bw_kernel<T, TW, VPL, NT><<<a.nblk, waves * 64, 0, a.stream>>>(
      static_cast<const T*>(a.dy), static_cast<const T*>(a.h), static_cast<const T*>(a.dh),
      static_cast<const TW*>(a.weight), a.eps, a.T, a.H, static_cast<T*>(a.dx), a.part);
}

// One chunk a lane up to 8 waves of bf16 and 16 of fp32 rows, then two.  With the
// reduction, us for one / two: bf16 4096 x 4096 29.4 / 30.9, 16384 x 4096 95 / 97, 8192 x
// 5120 80 / 85 (at the edge, where one would be faster), 1024 x 7168 23.1 / 21.9, 8192
// x 7168 98 / 92, 8192 x 8192 106 / 102; fp32 16384 x 1408 76 / 78, 8192 x 4096 107 / 109,
// 1024 x 7168 36 / 31, 8192 x 7168 206 / 187 (from about 7168 on two would be).  The
// two-chunk bf16 form fills 128 VGPRs and spills two or three of them.
template <typename T, typename TW> void bw_pick(const BwArgs& a) {
  const bool nt = static_cast<int64_t>(a.T) * a.H * static_cast<int64_t>(sizeof(T)) >= kStreamBytes;
  if (a.H <= 64 * 8 * (sizeof(T) == 4 ? 16 : 8)) nt ? bw_launch<T, TW, 1, true>(a) : bw_launch<T, TW, 1, false>(a);
  else nt ? bw_launch<T, TW, 2, true>(a) : bw_launch<T, TW, 2, false>(a);
}

inline bool norm_sizes(int T, int H) { return T >= 0 && H > 0; }
inline bool norm_limits(int T, int H) { return H % 8 == 0 && H <= kMaxH && T <= kMaxRows; }
inline bool good_eps(float eps) { return eps >= 0.f && eps < INFINITY; }

}  // namespace

extern "C" moe_status moe_add_rms_norm(const void* x, const void* residual, moe_dtype x_dt, const void* weight,
                                       moe_dtype w_dt, float eps, int T, int H, void* h_out, void* y, void* y8,
                                       float* y8_scales, hipStream_t stream) {
  MOE_CHECK(norm_sizes(T, H) && good_eps(eps), MOE_ERR_INVALID_ARG);
  MOE_CHECK(moe_host::valid_dtype(x_dt) && moe_host::valid_dtype(w_dt), MOE_ERR_INVALID_ARG);
  MOE_CHECK(real_dtype(x_dt) && real_dtype(w_dt), MOE_ERR_UNSUPPORTED);
  MOE_CHECK(norm_limits(T, H), MOE_ERR_UNSUPPORTED);
  MOE_CHECK(h_out || y || y8 || T == 0, MOE_ERR_INVALID_ARG);
  MOE_CHECK(!y8 == !y8_scales, MOE_ERR_INVALID_ARG);
  MOE_CHECK(!y8 || H % 128 == 0, MOE_ERR_UNSUPPORTED);
  if (T == 0) return MOE_OK;
  MOE_CHECK(x && weight && (!y || y != h_out), MOE_ERR_INVALID_ARG);
  MOE_CHECK(aligned16(x) && aligned16(residual) && aligned16(weight) && aligned16(h_out) && aligned16(y) && aligned16(y8),
            MOE_ERR_INVALID_ARG);
  return in_slices(T, kMaxWaves * 64, [&](int64_t t, int rows) {
    auto at = [&](auto* p, int64_t step) { return p ? p + t * step : p; };
    const int64_t bytes = static_cast<int64_t>(H) * (x_dt == MOE_BF16 ? 2 : 4);
    const FwArgs a{at(static_cast<const uint8_t*>(x), bytes), at(static_cast<const uint8_t*>(residual), bytes), weight,
                   eps, rows, H, at(static_cast<uint8_t*>(h_out), bytes), at(static_cast<uint8_t*>(y), bytes),
                   at(static_cast<uint8_t*>(y8), H), at(y8_scales, H / 128), stream};
    if (x_dt == MOE_BF16) {
      if (w_dt == MOE_BF16) fw_pick<uint16_t, uint16_t>(a);
      else fw_pick<uint16_t, float>(a);
    } else {
      if (w_dt == MOE_BF16) fw_pick<float, uint16_t>(a);
      else fw_pick<float, float>(a);
    }
  });
}

extern "C" size_t moe_add_rms_norm_backward_workspace_bytes(int T, int H) {
  if (!norm_sizes(T, H) || !norm_limits(T, H)) return 0;
  return static_cast<size_t>(bw_blocks(T, H)) * H * sizeof(float);
}

extern "C" moe_status moe_add_rms_norm_backward(const void* dy, const void* h, const void* dh, moe_dtype dt,
                                                const void* weight, moe_dtype w_dt, float eps, int T, int H,
                                                void* dx, float* d_weight, void* workspace, size_t workspace_bytes,
                                                hipStream_t stream) {
  MOE_CHECK(norm_sizes(T, H) && good_eps(eps), MOE_ERR_INVALID_ARG);
  MOE_CHECK(moe_host::valid_dtype(dt) && moe_host::valid_dtype(w_dt), MOE_ERR_INVALID_ARG);
  MOE_CHECK(real_dtype(dt) && real_dtype(w_dt), MOE_ERR_UNSUPPORTED);
  MOE_CHECK(norm_limits(T, H), MOE_ERR_UNSUPPORTED);
  MOE_CHECK(d_weight && aligned16(d_weight), MOE_ERR_INVALID_ARG);
  const size_t need = moe_add_rms_norm_backward_workspace_bytes(T, H);
  if (T > 0) {
    MOE_CHECK(dy && h && weight && dx && workspace, MOE_ERR_INVALID_ARG);
    MOE_CHECK(aligned16(dy) && aligned16(h) && aligned16(dh) && aligned16(weight) && aligned16(dx) && aligned16(workspace),
              MOE_ERR_INVALID_ARG);
    MOE_CHECK(workspace_bytes >= need, MOE_ERR_WORKSPACE);
    const BwArgs a{dy, h, dh, weight, eps, T, H, dx, static_cast<float*>(workspace), bw_blocks(T, H), stream};
    if (dt == MOE_BF16) {
      if (w_dt == MOE_BF16) bw_pick<uint16_t, uint16_t>(a);
      else bw_pick<uint16_t, float>(a);
    } else {
      if (w_dt == MOE_BF16) bw_pick<float, uint16_t>(a);
      else bw_pick<float, float>(a);
    }
    MOE_LAUNCH_CHECK();
  }
  const int nblk = T > 0 ? bw_blocks(T, H) : 0, grid = (H + kRedCols - 1) / kRedCols;
  const float* part = static_cast<const float*>(workspace);
  if (nblk <= 1024) reduce_dw_kernel<32><<<grid, 256, 0, stream>>>(part, nblk, H, d_weight);
  else reduce_dw_kernel<128><<<grid, 1024, 0, stream>>>(part, nblk, H, d_weight);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}
