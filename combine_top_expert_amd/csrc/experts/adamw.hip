// moe_adamw_step: one AdamW update of many tensors, states in 32 or in 8 bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p - lr wd p - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every element is read and written once.  The tensors of a call are listed in
// the kernel's arguments (no table on the device, so a captured call carries its
// own), a workgroup takes neighbouring elements of one of them, and a lane four at
// a time: each load of a wave is one contiguous KB of fp32.
//
// 8-bit states are e4m3 codes with one scale per 128 elements: half a wave
// holds such a block, so its maximum takes four DPP moves and one exchange.
// v is kept as its root, whose exponents span half as many powers of two.
//
// Bound by memory: 30 bytes an element with bf16 weights, fp32 masters, gradients
// and states, 18 with 8-bit states.  277 M elements take 1345 us (6.2 TB/s) and 836 us
// (6.0 TB/s; about 80 vector instructions an element, a quarter of them the random bits),
// with lr and step on the device 2 % more and the same.  160 tensors of 1.8 to 12.5 K elements, 13.7 us,
// are two launches that each begin with a chain of scalar loads.
// Loads and stores are non-temporal (1550 us through the caches).

#include <math.h>

#include "experts_common.h"

namespace {

using namespace moe_experts;

constexpr int kThreads = 256;
// Groups of four elements a lane takes: one with fp32 states (bf16 weights, fp32 masters and gradients,
// 277 M elements: 1347 us against 1450 with 2 or 4), four with 8-bit ones.
constexpr int steps_of(bool s8) { return s8 ? 4 : 1; }
constexpr int span_of(bool s8) { return kThreads * 4 * steps_of(s8); }    // elements of a workgroup
constexpr int kMaxBlocks = 1 << 22;                // of one launch
constexpr int kUnit = 4096;                        // parts of a tensor begin at multiples of it

// Tensors, or parts of at most 2^30 elements of them, of one launch: as many as the 4 KB of a kernel's
// arguments hold beside the configuration.
template <bool S8, bool MASTER> struct Batch {
  static constexpr int kTensors = 3840 / (48 + (S8 ? 16 : 0) + (MASTER ? 8 : 0));
  void* param[kTensors];
  const void* grad[kTensors];
  void* m[kTensors];
  void* v[kTensors];
  float* master[MASTER ? kTensors : 1];
  float* ms[S8 ? kTensors : 1];
  float* vs[S8 ? kTensors : 1];
  int32_t n[kTensors];                             // elements
  int32_t first[kTensors];                         // index of the first in its tensor, in units of kUnit
  int32_t begin[kTensors];                         // first workgroup
  int32_t tensor[kTensors];
  int count;
};

struct Config {
  float b1, a1, b2, a2, eps;                       // a1 = 1 - b1, a2 = 1 - b2
  float rate, decay, root2;                        // unit lr / (1 - b1^t), lr wd, unit / sqrt(1 - b2^t)
  float unit;                                      // of the quotient's denominator (eps times it, too): a power of two
  double lr, wd, d1, d2, inv1;                     // for numbers on the device: b1, b2, 1 / (1 - b1^t)
  uint32_t seed, step;                             // step's low 32 bits
  const float* lr_device;
  const int64_t* step_device;
  const float* grad_scale;
};

__host__ __device__ inline uint32_t mix(uint32_t x) {
  x = (x ^ x >> 16) * 0x9e3779b9u;
  x = (x ^ x >> 15) * 0xbb67ae85u;
  return x ^ x >> 16;
}

// b^t in fp64 by squaring (t >= 1)
__device__ __forceinline__ double power(double b, int64_t t) {
  double r = 1.0;
  for (; t; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}

// ---------------------------------------------------------------- four neighbouring elements

template <typename T> struct Four;
template <> struct Four<float> {
  static __device__ __forceinline__ void load(const void* p, int64_t i, int left, float (&v)[4]) {
    const float* q = static_cast<const float*>(p) + i;
    if (left >= 4) {
      const uint4 r = moe::load_nt16(q);
      v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = k < left ? q[k] : 0.f;
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, int left, const float (&v)[4]) {
    float* q = static_cast<float*>(p) + i;
    if (left >= 4) {
      moe::store_nt16(q, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                    __float_as_uint(v[3])));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < left) q[k] = v[k];
    }
  }
};
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
template <> struct Four<uint16_t> {                // bf16
  static __device__ __forceinline__ void load(const void* p, int64_t i, int left, float (&v)[4]) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (left >= 4) {
      const u32x2_t r = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(q));
      v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xffff0000u);
      v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xffff0000u);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = k < left ? moe::bf16_to_f32(q[k]) : 0.f;
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, int left, const float (&v)[4]) {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    uint16_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = moe::f32_to_bf16(v[k]);
    if (left >= 4) {
      const u32x2_t r = {static_cast<uint32_t>(h[0]) | static_cast<uint32_t>(h[1]) << 16,
                         static_cast<uint32_t>(h[2]) | static_cast<uint32_t>(h[3]) << 16};
      __builtin_nontemporal_store(r, reinterpret_cast<u32x2_t*>(q));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < left) q[k] = h[k];
    }
  }
};

// e4m3 codes of four elements
__device__ __forceinline__ uint32_t load_codes(const void* p, int64_t i, int left) {
  const uint8_t* q = static_cast<const uint8_t*>(p) + i;
  if (left >= 4) return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(q));
  uint32_t r = 0;
  for (int k = 0; k < 4; ++k)
    if (k < left) r |= static_cast<uint32_t>(q[k]) << (8 * k);
  return r;
}
__device__ __forceinline__ void store_codes(void* p, int64_t i, int left, uint32_t c) {
  uint8_t* q = static_cast<uint8_t*>(p) + i;
  if (left >= 4) {
    __builtin_nontemporal_store(c, reinterpret_cast<uint32_t*>(q));
  } else {
    for (int k = 0; k < 4; ++k)
      if (k < left) q[k] = static_cast<uint8_t>(c >> (8 * k));
  }
}
__device__ __forceinline__ void decode(uint32_t c, float scale, float (&v)[4]) {
  v[0] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(c), 0) * scale;
  v[1] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(c), 1) * scale;
  v[2] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(c), 2) * scale;
  v[3] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(c), 3) * scale;
}

// ---------------------------------------------------------------- rounding to 8 bits

// y, |y| <= 448, to a value that e4m3 holds.  Between two of them lie 20 bits of
// y's fraction (below 2^-6, where the step no longer shrinks, 2^-6 is added so
// that the same 20 bits stand there): 16 random bits are added to their upper
// ones, and the carry rounds up.
__device__ __forceinline__ float to_code_value(float y, uint32_t bits16) {
  const float a = fabsf(y);
  const float off = a < 0x1p-6f ? 0x1p-6f : 0.f;
  const float t = __uint_as_float((__float_as_uint(a + off) + (bits16 << 4)) & 0xfff00000u) - off;
  return copysignf(t, y);
}

// The largest finite magnitude of a block of 128: lanes 0..31 or 32..63 of the wave.  ALL: also of those that
// are not finite (NaN above infinity), as bits.
template <bool ALL> __device__ __forceinline__ uint32_t block_bits(const float (&x)[4]) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t b = magnitude(x[k]);
    top = max(top, ALL || b < 0x7f800000u ? b : 0u);
  }
  top = dpp_max<kMirror>(dpp_max<kHalfMirror>(dpp_max<kXor2>(dpp_max<kXor1>(top))));
  const uint32_t other = static_cast<uint32_t>(__builtin_amdgcn_ds_swizzle(static_cast<int>(top), 0x401f));  // lane ^ 16
  return max(top, other);
}
__device__ __forceinline__ float block_max(uint32_t bits) {
  const float f = __uint_as_float(bits);
  return f < 1e-30f ? 0.f : f;
}

// four values to codes, with random bits taken from r[k] >> SHIFT; LEAST: what
// is not zero does not become zero; BROKEN: some of them may not be finite
template <int SHIFT, bool LEAST, bool BROKEN>
__device__ __forceinline__ uint32_t encode(const float (&x)[4], float top, const uint32_t (&r)[4]) {
  const float inv = top > 0.f ? 448.f / top : 0.f;
  float y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float s = x[k] * inv;
    y[k] = to_code_value(__builtin_amdgcn_fmed3f(s, -448.f, 448.f), r[k] >> SHIFT & 0xffffu);
    if (LEAST && y[k] == 0.f && s > 0.f) y[k] = 0x1p-9f;
    if (BROKEN && !(magnitude(x[k]) < 0x7f800000u)) y[k] = __uint_as_float(0x7fc00000u);
  }
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  c = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
  return static_cast<uint32_t>(c);
}
// a block's state: codes of four elements, and its scale's maximum
template <int SHIFT, bool LEAST>
__device__ __forceinline__ uint32_t encode_block(const float (&x)[4], const uint32_t (&r)[4], float& top) {
  const uint32_t bits = block_bits<true>(x);
  if (__ballot(bits >= 0x7f800000u)) {             // seldom: something of the wave's is not finite
    top = block_max(block_bits<false>(x));
    return encode<SHIFT, LEAST, true>(x, top, r);
  }
  top = block_max(bits);
  return encode<SHIFT, LEAST, false>(x, top, r);
}

// ---------------------------------------------------------------- the step

template <typename TP, typename TG, bool S8, bool MASTER>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Batch<S8, MASTER> b, const Config c) {
  constexpr int kSteps = steps_of(S8);
  // the last part that begins at or before this workgroup
  int lo = 0, hi = b.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.begin[mid] <= static_cast<int>(blockIdx.x)) lo = mid;
    else hi = mid - 1;
  }
  const int n = b.n[lo];
  const int base = (static_cast<int>(blockIdx.x) - b.begin[lo]) * span_of(S8);
  const void* gp = b.grad[lo];
  void* mp = b.m[lo];
  void* vp = b.v[lo];
  void* pp = b.param[lo];
  float* wp = MASTER ? b.master[lo] : nullptr;

  float g[kSteps][4], w[kSteps][4], m[kSteps][4], v[kSteps][4];
  uint32_t mc[kSteps], vc[kSteps];
  float mk[kSteps], vk[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int i = base + u * (kThreads * 4) + static_cast<int>(threadIdx.x) * 4;
    const int left = n - i < 4 ? (n - i < 0 ? 0 : n - i) : 4;
    Four<TG>::load(gp, i, left, g[u]);
    if constexpr (MASTER) Four<float>::load(wp, i, left, w[u]);
    else Four<TP>::load(pp, i, left, w[u]);
    if constexpr (S8) {
      mc[u] = load_codes(mp, i, left);
      vc[u] = load_codes(vp, i, left);
      mk[u] = left ? b.ms[lo][i >> 7] : 0.f;
      vk[u] = left ? b.vs[lo][i >> 7] : 0.f;
    } else {
      Four<float>::load(mp, i, left, m[u]);
      Four<float>::load(vp, i, left, v[u]);
    }
  }

  float rate = c.rate, decay = c.decay, root2 = c.root2, gs = 1.f;
  uint32_t step = c.step;
  if (c.grad_scale) {
    gs = *c.grad_scale;
    if (!(magnitude(gs) < 0x7f800000u)) return;    // a step to be skipped
  }
  if (c.step_device || c.lr_device) {
    const int64_t t = c.step_device ? *c.step_device : 1;
    if (t < 1) return;
    // one wave of the workgroup works the numbers out for all
    __shared__ float shared[3];
    if (threadIdx.x < MOE_WAVE) {
      const double lr = c.lr_device ? static_cast<double>(*c.lr_device) : c.lr;
      const double inv1 = c.step_device ? 1.0 / (1.0 - power(c.d1, t)) : c.inv1;
      const double p2 = c.step_device ? power(c.d2, t) : 0.0;
      if (threadIdx.x == 0) {
        shared[0] = static_cast<float>(lr * inv1) * c.unit;
        shared[1] = static_cast<float>(lr * c.wd);
        shared[2] = c.step_device ? static_cast<float>(1.0 / sqrt(1.0 - p2)) * c.unit : c.root2;
      }
    }
    __syncthreads();
    rate = shared[0], decay = shared[1], root2 = shared[2];
    if (c.step_device) step = static_cast<uint32_t>(t);
  }
  const uint32_t key = S8 ? mix(mix(mix(c.seed) + step) + static_cast<uint32_t>(b.tensor[lo])) : 0u;

#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int i = base + u * (kThreads * 4) + static_cast<int>(threadIdx.x) * 4;
    const int left = n - i < 4 ? (n - i < 0 ? 0 : n - i) : 4;
    if constexpr (S8) {
      decode(mc[u], mk[u], m[u]);
      decode(vc[u], vk[u], v[u]);
    }
    float r[4];                                    // sqrt(v)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
// each operation of the states rounds once: one that is rounded to 8 bits next to a border is then the same
// for everyone who computes it in fp32.  The update's quotient takes the hardware's reciprocal (1 ulp), of a
// denominator that the unit keeps in its range.
#pragma clang fp contract(off)
      const float gk = g[u][k] * gs;
      m[u][k] = c.b1 * m[u][k] + c.a1 * gk;
      const float old = S8 ? v[u][k] * v[u][k] : v[u][k];
      v[u][k] = c.b2 * old + c.a2 * (gk * gk);
      r[k] = sqrtf(v[u][k]);
      w[u][k] = w[u][k] - decay * w[u][k] - rate * (m[u][k] * __builtin_amdgcn_rcpf(r[k] * root2 + c.eps));
    }
    if constexpr (S8) {
      // elements behind the tensor's end are zeros here and change no maximum
      uint32_t random[4];
      const uint64_t at = static_cast<uint64_t>(b.first[lo]) * kUnit + static_cast<uint32_t>(i);
      const uint32_t k2 = at >> 32 ? mix(key + static_cast<uint32_t>(at >> 32)) : key;
#pragma unroll
      for (int k = 0; k < 4; ++k) random[k] = mix((static_cast<uint32_t>(at) + k) ^ k2);
      float mt, rt;
      store_codes(mp, i, left, encode_block<16, false>(m[u], random, mt));
      store_codes(vp, i, left, encode_block<0, true>(r, random, rt));
      if ((threadIdx.x & 31) == 0 && left) {
        b.ms[lo][i >> 7] = mt * (1.f / 448.f);
        b.vs[lo][i >> 7] = rt * (1.f / 448.f);
      }
    } else {
      Four<float>::store(mp, i, left, m[u]);
      Four<float>::store(vp, i, left, v[u]);
    }
    if constexpr (MASTER) Four<float>::store(wp, i, left, w[u]);
    Four<TP>::store(pp, i, left, w[u]);
  }
}

template <typename TP, typename TG, bool S8, bool MASTER>
moe_status run(const moe_adamw_tensor* tensors, int count, const Config& c, hipStream_t stream) {
  constexpr int span = span_of(S8), sb = S8 ? 1 : 4;
  Batch<S8, MASTER> b;
  static_assert(sizeof(b) + sizeof(c) <= 4096, "a kernel's arguments");
  int blocks = 0;
  b.count = 0;
  auto flush = [&]() {
    if (!b.count) return true;
    adamw_kernel<TP, TG, S8, MASTER><<<blocks, kThreads, 0, stream>>>(b, c);
    blocks = b.count = 0;
    return hipGetLastError() == hipSuccess;
  };
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    for (int64_t at = 0; at < t.n;) {
      int64_t most = static_cast<int64_t>(kMaxBlocks - blocks) * span / kUnit * kUnit;
      if (b.count == b.kTensors || most == 0) {
        if (!flush()) return MOE_ERR_HIP;
        most = static_cast<int64_t>(kMaxBlocks) * span;
      }
      most = most < 1 << 30 ? most : 1 << 30;
      const int64_t n = t.n - at < most ? t.n - at : most;
      const int k = b.count++;
      b.param[k] = static_cast<TP*>(t.param) + at;
      b.grad[k] = static_cast<const TG*>(t.grad) + at;
      b.m[k] = static_cast<uint8_t*>(t.exp_avg) + at * sb;
      b.v[k] = static_cast<uint8_t*>(t.exp_avg_sq) + at * sb;
      if constexpr (MASTER) b.master[k] = t.master + at;
      if constexpr (S8) b.ms[k] = t.exp_avg_scale + at / 128, b.vs[k] = t.exp_avg_sq_scale + at / 128;
      b.n[k] = static_cast<int32_t>(n), b.first[k] = static_cast<int32_t>(at / kUnit);
      b.begin[k] = blocks, b.tensor[k] = i;
      blocks += static_cast<int>((n + span - 1) / span);
      at += n;
    }
  }
  return flush() ? MOE_OK : MOE_ERR_HIP;
}

template <typename TP, typename TG>
moe_status run(const moe_adamw_tensor* tensors, int count, const Config& c, bool s8, bool master, hipStream_t stream) {
  if constexpr (sizeof(TP) == 2)
    if (master)
      return s8 ? run<TP, TG, true, true>(tensors, count, c, stream) : run<TP, TG, false, true>(tensors, count, c, stream);
  return s8 ? run<TP, TG, true, false>(tensors, count, c, stream) : run<TP, TG, false, false>(tensors, count, c, stream);
}

bool rate_ok(double v) { return v >= 0.0 && v < INFINITY; }        // and no NaN
bool beta_ok(double v) { return v >= 0.0 && v < 1.0; }

}  // namespace

extern "C" moe_status moe_adamw_step(const moe_adamw_tensor* tensors, int count, moe_dtype p_dt, moe_dtype g_dt,
                                     moe_dtype s_dt, const moe_adamw_config* config, hipStream_t stream) {
  MOE_CHECK(count >= 0 && config, MOE_ERR_INVALID_ARG);
  MOE_CHECK(moe_host::valid_dtype(p_dt) && moe_host::valid_dtype(g_dt) && moe_host::valid_dtype(s_dt),
            MOE_ERR_INVALID_ARG);
  MOE_CHECK(real_dtype(p_dt) && real_dtype(g_dt) && s_dt != MOE_BF16, MOE_ERR_UNSUPPORTED);
  const moe_adamw_config& f = *config;
  MOE_CHECK(rate_ok(f.lr) && rate_ok(f.eps) && rate_ok(f.weight_decay) && beta_ok(f.beta1) && beta_ok(f.beta2),
            MOE_ERR_INVALID_ARG);
  MOE_CHECK(f.step_device || f.step >= 1, MOE_ERR_INVALID_ARG);
  MOE_CHECK(aligned(f.lr_device, 4) && aligned(f.grad_scale, 4) && aligned(f.step_device, 8), MOE_ERR_INVALID_ARG);
  if (count == 0) return MOE_OK;
  MOE_CHECK(tensors, MOE_ERR_INVALID_ARG);
  const bool s8 = s_dt == MOE_FP8_E4M3;
  bool master = false;                             // of the tensors with elements: for all or for none
  for (int i = 0; i < count; ++i) master = master || (tensors[i].n > 0 && tensors[i].master);
  MOE_CHECK(!master || p_dt == MOE_BF16, MOE_ERR_UNSUPPORTED);
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    MOE_CHECK(t.n >= 0, MOE_ERR_INVALID_ARG);
    MOE_CHECK(t.n <= 1ll << 40, MOE_ERR_UNSUPPORTED);
    if (t.n == 0) continue;
    MOE_CHECK(t.param && t.grad && t.exp_avg && t.exp_avg_sq && (t.master != nullptr) == master, MOE_ERR_INVALID_ARG);
    MOE_CHECK((t.exp_avg_scale != nullptr) == s8 && (t.exp_avg_sq_scale != nullptr) == s8, MOE_ERR_INVALID_ARG);
    MOE_CHECK(aligned(t.param, 16) && aligned(t.master, 16) && aligned(t.grad, 16) && aligned(t.exp_avg, 16) &&
                  aligned(t.exp_avg_sq, 16) && aligned(t.exp_avg_scale, 4) && aligned(t.exp_avg_sq_scale, 4),
              MOE_ERR_INVALID_ARG);
  }
  Config c{};
  // The denominator, at least eps and at most 2^64 / sqrt(2^-53) + eps, in a unit that makes it a normal number with a
  // normal reciprocal also where eps itself is not one; 1 for any usual eps.
  c.unit = f.eps < 0x1p-100 ? 0x1p32f : f.eps > 0x1p100 ? 0x1p-32f : 1.f;
  c.eps = static_cast<float>(f.eps * c.unit);
  if (f.eps > 0.0 && c.eps < 0x1p-117f) c.eps = 0x1p-117f;           // 2^-149 in the unit: fp32's least number
  c.lr = f.lr, c.wd = f.weight_decay;
  c.b1 = static_cast<float>(f.beta1), c.a1 = static_cast<float>(1.0 - f.beta1);
  c.b2 = static_cast<float>(f.beta2), c.a2 = static_cast<float>(1.0 - f.beta2);
  c.d1 = f.beta1, c.d2 = f.beta2;
  c.seed = f.seed;
  c.lr_device = f.lr_device, c.step_device = f.step_device, c.grad_scale = f.grad_scale;
  if (!f.step_device) {
    c.step = static_cast<uint32_t>(f.step);
    c.inv1 = 1.0 / (1.0 - pow(f.beta1, static_cast<double>(f.step)));
    c.root2 = static_cast<float>(1.0 / sqrt(1.0 - pow(f.beta2, static_cast<double>(f.step)))) * c.unit;
    c.rate = static_cast<float>(f.lr * c.inv1) * c.unit;
    c.decay = static_cast<float>(f.lr * f.weight_decay);
  }
  if (p_dt == MOE_F32)
    return g_dt == MOE_F32 ? run<float, float>(tensors, count, c, s8, master, stream)
                           : run<float, uint16_t>(tensors, count, c, s8, master, stream);
  return g_dt == MOE_F32 ? run<uint16_t, float>(tensors, count, c, s8, master, stream)
                         : run<uint16_t, uint16_t>(tensors, count, c, s8, master, stream);
}
