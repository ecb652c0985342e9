// moe_router_group_topk and its backward.
//
// One wavefront per token; lane l holds experts l, l + 64, ...  A score c =
// s + bias is held as the order-preserving 32-bit key of the router's top-K
// (NaN lowest among the live, 0 for a masked or retired entry), so a selection
// round is a wave maximum and a ballot for its lowest holder.
//
// The order is the one of exact scores.  Without a bias it is the logits' order,
// which needs no arithmetic.  Where arithmetic decides (a bias, or the sums that
// rank the groups), an fp32 score is off by at most kRel 2^-24 of the row's
// largest score plus the rounding of the bias's addition; a row in which two
// neighbours of the order lie within that of each other is decided again by
// the same wave in fp64 (route_exact).

#include "block_common.h"
#include "router_common.h"

namespace {

using namespace moe_block;
using moe_router::score_key;
using moe_router::wave_max_f32;
using moe_router::wave_max_u32;
using moe_router::wave_sum_f32;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / MOE_WAVE;
constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr float kMask = -3.3e38f;   // covers -inf and the lowest finite fp32 and bf16
// expf 1 ulp, the sum of the softmax (64 lanes x 16 terms, a tree: 22
// roundings of positive terms), l - max one rounding whose effect on e is at
// most 0.37 2^-24 of the largest e, one addition and one division: below 28
// half-ulps.
constexpr float kRel = 32.0f * 5.9604644775390625e-8f;

struct RouteArgs {
  const float* logits;
  const float* bias;
  int T, E, K;
  int sigmoid;
  int n_group, topk_group, group_top, group_size;
  int renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

__device__ __forceinline__ float sigmoid_f(float l) { return 1.0f / (1.0f + expf(-l)); }

// value of a key made by score_key (keys above 1)
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k <= 1u) return k ? NAN : -INFINITY;
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// wave maximum of a double, NaN ignored by the caller's mapping
__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmax(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

constexpr double kDead = -INFINITY;
constexpr double kNan = -1e300;      // where a NaN score ranks

// The choice in fp64: lane k returns round k's expert (or -1).  `c` is the
// wave's LDS row of E doubles.
__device__ __noinline__ int route_exact(const RouteArgs& a, const float* __restrict__ row, double* c, int lane) {
  double m = kDead, sum = 0.0;
  if (!a.sigmoid) {
    for (int e = lane; e < a.E; e += MOE_WAVE)
      if (!(row[e] <= kMask)) m = fmax(m, static_cast<double>(row[e]));
    m = wave_max_f64(m);
    for (int e = lane; e < a.E; e += MOE_WAVE)
      if (!(row[e] <= kMask)) sum += exp(static_cast<double>(row[e]) - m);
    sum = wave_sum_f64(sum);
  }
  for (int e = lane; e < a.E; e += MOE_WAVE) {
    const double l = row[e];
    double v = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - m) / sum;
    const bool dead = row[e] <= kMask || (a.bias && a.bias[e] <= kMask);
    if (a.bias) v += static_cast<double>(a.bias[e]);
    c[e] = dead ? kDead : (v != v ? kNan : v);
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  uint64_t keep = ~0ull;
  if (a.n_group > 1) {
    double gs = kDead;
    if (lane < a.n_group) {
      double t1 = kDead, t2 = kDead;
      for (int i = 0; i < a.group_size; ++i) {
        const double v = c[lane * a.group_size + i];
        if (v > t1) { t2 = t1; t1 = v; }
        else if (v > t2) t2 = v;
      }
      gs = (a.group_top == 2 && t2 != kDead) ? t1 + t2 : t1;
      if (t1 == kNan || (a.group_top == 2 && t2 == kNan)) gs = kNan;
    }
    keep = 0;
    for (int g = 0; g < a.topk_group; ++g) {
      const bool in = lane < a.n_group && !((keep >> lane) & 1);
      const double best = wave_max_f64(in ? gs : kDead);
      const uint64_t holders = __ballot(in && gs == best);
      if (!holders) break;
      keep |= holders & (~holders + 1);
    }
  }
  int my = -1;
  for (int k = 0; k < a.K; ++k) {
    double best = kDead;
    int be = 0x7fffffff;
    for (int e = lane; e < a.E; e += MOE_WAVE) {
      const double v = c[e];
      if (v > best && ((keep >> (a.n_group > 1 ? e / a.group_size : 0)) & 1)) { best = v; be = e; }
    }
    const double win = wave_max_f64(best);
    int e = (win != kDead && best == win) ? be : 0x7fffffff;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) e = min(e, __shfl_xor(e, d));
    if (e == 0x7fffffff) break;
    if ((e & 63) == lane) c[e] = kDead;
    if (lane == k) my = e;
  }
  return my;
}

template <int NPL>   // scores per lane: E <= 64 * NPL
__global__ __launch_bounds__(kThreads) void group_topk_kernel(RouteArgs a) {
  extern __shared__ double lds[];
  const int lane = moe::lane_id();
  const int wave = threadIdx.x >> 6;
  const int t = blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  const float* row = a.logits + static_cast<int64_t>(t) * a.E;
  double* c64 = lds + static_cast<size_t>(wave) * a.E;
  float* c32 = reinterpret_cast<float*>(c64);

  float l[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const int e = lane + MOE_WAVE * j;
    l[j] = e < a.E ? row[e] : -INFINITY;
  }
  float m = 0.f, sum = 1.f;
  if (!a.sigmoid) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (!(l[j] <= kMask)) m = fmaxf(m, l[j]);
    m = wave_max_f32(m);
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (!(l[j] <= kMask)) sum += expf(l[j] - m);
    sum = wave_sum_f32(sum);
  }
  auto score = [&](float x) { return a.sigmoid ? sigmoid_f(x) : (x <= kMask ? 0.f : expf(x - m) / sum); };

  // keys: of the logits without a bias, of c with one
  uint32_t key[NPL];
  float smax = 0.f, cmax = 0.f;
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const int e = lane + MOE_WAVE * j;
    key[j] = 0;
    if (e < a.E && !(l[j] <= kMask)) {
      float v = l[j];
      if (a.bias) {
        const float b = a.bias[e], s = score(l[j]);
        v = s + b;
        if (!(b <= kMask)) {
          key[j] = max(score_key(v), 1u);
          smax = fmaxf(smax, s);
          if (fabsf(v) < INFINITY) cmax = fmaxf(cmax, fabsf(v));
        }
      } else {
        key[j] = (sum != sum) ? 1u : max(score_key(v), 1u);
      }
    }
  }
  // how far an fp32 c may be off (0 without a bias: logits are exact)
  float tol = 0.f;
  if (a.bias) tol = kRel * wave_max_f32(smax) + 1.2e-7f * wave_max_f32(cmax);

  bool near = false;
  if (a.n_group > 1) {
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      const int e = lane + MOE_WAVE * j;
      if (e < a.E) c32[e] = __uint_as_float(key[j]);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    uint32_t gkey = 0;
    float gs = -INFINITY;
    if (lane < a.n_group) {
      uint32_t k1 = 0, k2 = 0;
      for (int i = 0; i < a.group_size; ++i) {
        const uint32_t k = __float_as_uint(c32[lane * a.group_size + i]);
        k2 = max(k2, min(k1, k));
        k1 = max(k1, k);
      }
      if (k1) {
        const bool two = a.group_top == 2 && k2;
        gs = key_value(k1);
        if (!a.bias && a.group_top == 2) gs = score(gs);
        if (two) gs += a.bias ? key_value(k2) : score(key_value(k2));
        gkey = max(score_key(gs), 1u);
      }
    }
    uint64_t keep = 0;
    float last = 0.f;
    for (int g = 0; g <= a.topk_group; ++g) {
      const bool in = lane < a.n_group && !((keep >> lane) & 1);
      const uint32_t win = wave_max_u32(in ? gkey : 0u);
      const uint64_t holders = __ballot(in && gkey == win);
      if (!holders || win == 0) break;
      const float v = key_value(win);
      if (g == a.topk_group) {      // the best group that stays out
        // without a bias a group's sum is off by kRel of itself (1e-37: what
        // fp32 loses below its normal range); a single logit is exact
        if (a.bias) near = last - v <= 4.f * tol;
        else if (a.group_top == 2) near = last - v <= kRel * (last + v) + 1e-37f;
        break;
      }
      keep |= holders & (~holders + 1);
      last = v;
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      const int e = lane + MOE_WAVE * j;
      if (e < a.E && !((keep >> (e / a.group_size)) & 1)) key[j] = 0;
    }
  }

  int my = -1;
  float last = INFINITY;
  if (!near) {
    for (int k = 0; k <= a.K; ++k) {
      uint32_t best = 0;
#pragma unroll
      for (int j = 0; j < NPL; ++j) best = max(best, key[j]);
      const uint32_t win = wave_max_u32(best);
      if (win == 0) break;
      const float v = key_value(win);
      if (a.bias && last - v <= 2.f * tol) { near = true; break; }
      if (k == a.K) break;
      last = v;
      int e = -1;
#pragma unroll
      for (int j = 0; j < NPL; ++j) {
        const uint64_t holders = __ballot(key[j] == win);
        if (e < 0 && holders) {
          const int owner = __builtin_ctzll(holders);
          e = MOE_WAVE * j + owner;
          if (lane == owner) key[j] = 0;
        }
      }
      if (lane == k) my = e;
    }
  }
  if (near) my = route_exact(a, row, c64, lane);

  float w = 0.f;
  if (lane < a.K && my >= 0) w = score(row[my]);
  if (a.renorm) w = w / (wave_sum_f32(w) + 1e-20f);
  if (lane < a.K) {
    a.ids[static_cast<int64_t>(t) * a.K + lane] = my;
    a.weights[static_cast<int64_t>(t) * a.K + lane] = my >= 0 ? w * a.scale : 0.f;
  }
}

// Backward: one wavefront per token.  Lane k holds route k's id, score and
// ds; the row's other elements are 0 (sigmoid) or the softmax's -s_e dot.
template <int NPL>
__global__ __launch_bounds__(kThreads) void group_topk_bw_kernel(RouteArgs a, const float* __restrict__ d_weights,
                                                                 float* __restrict__ d_logits) {
  const int lane = moe::lane_id();
  const int t = blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const float* row = a.logits + static_cast<int64_t>(t) * a.E;
  float l[NPL];
  float m = 0.f, sum = 1.f;
  if (!a.sigmoid) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      const int e = lane + MOE_WAVE * j;
      l[j] = e < a.E ? row[e] : -INFINITY;
      if (!(l[j] <= kMask)) m = fmaxf(m, l[j]);
    }
    m = wave_max_f32(m);
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      l[j] = l[j] <= kMask ? 0.f : expf(l[j] - m);
      sum += l[j];
    }
    sum = wave_sum_f32(sum);
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < NPL; ++j) l[j] *= inv;      // s
  }
  int id = lane < a.K ? a.ids[static_cast<int64_t>(t) * a.K + lane] : -1;
  if (id >= a.E) id = -1;
  float s = 0.f, d = 0.f;
  if (id >= 0) {
    const float x = row[id];
    if (!(x <= kMask)) s = a.sigmoid ? sigmoid_f(x) : expf(x - m) / sum;
    d = d_weights[static_cast<int64_t>(t) * a.K + lane] * a.scale;
  }
  if (a.renorm) {
    const float S = wave_sum_f32(s) + 1e-20f;
    const float dot = wave_sum_f32(d * s) / S;
    d = id >= 0 ? (d - dot) / S : 0.f;
  }
  // g: what route k adds to its expert's element
  const float dot = a.sigmoid ? 0.f : wave_sum_f32(d * s);
  const float g = a.sigmoid ? d * s * (1.0f - s) : d * s;
  float o[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) o[j] = a.sigmoid ? 0.f : -l[j] * dot;
  for (int k = 0; k < a.K; ++k) {
    const int e = __builtin_amdgcn_readlane(id, k);
    if (e < 0) continue;
    const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), k));
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (e == lane + MOE_WAVE * j) o[j] += v;
  }
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const int e = lane + MOE_WAVE * j;
    if (e < a.E) d_logits[static_cast<int64_t>(t) * a.E + e] = o[j];
  }
}

template <int NPL> void launch_fw(const RouteArgs& a, hipStream_t stream) {
  const int grid = (a.T + kWaves - 1) / kWaves;
  group_topk_kernel<NPL><<<grid, kThreads, static_cast<size_t>(kWaves) * a.E * sizeof(double), stream>>>(a);
}
template <int NPL> void launch_bw(const RouteArgs& a, const float* dw, float* dl, hipStream_t stream) {
  group_topk_bw_kernel<NPL><<<(a.T + kWaves - 1) / kWaves, kThreads, 0, stream>>>(a, dw, dl);
}

}  // namespace

extern "C" moe_status moe_router_group_topk(const float* logits, const float* bias, int T, int E, int K,
                                            moe_score score, int n_group, int topk_group, int group_top, int renorm,
                                            float route_scale, int32_t* topk_ids, float* topk_weights,
                                            hipStream_t stream) {
  MOE_CHECK(T >= 0 && E >= 1 && K >= 1 && K <= E, MOE_ERR_INVALID_ARG);
  MOE_CHECK(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID, MOE_ERR_INVALID_ARG);
  MOE_CHECK(n_group >= 1 && n_group <= E && topk_group >= 1 && topk_group <= n_group, MOE_ERR_INVALID_ARG);
  MOE_CHECK(group_top == 1 || group_top == 2, MOE_ERR_INVALID_ARG);
  MOE_CHECK(E <= kMaxE && K <= kMaxK && n_group <= MOE_WAVE && E % n_group == 0, MOE_ERR_UNSUPPORTED);
  MOE_CHECK(K <= topk_group * (E / n_group), MOE_ERR_INVALID_ARG);
  MOE_CHECK(route_scale == route_scale && fabsf(route_scale) < INFINITY, MOE_ERR_INVALID_ARG);
  if (T == 0) return MOE_OK;
  MOE_CHECK(logits && topk_ids && topk_weights, MOE_ERR_INVALID_ARG);
  const RouteArgs a{logits, bias, T, E, K, score == MOE_SCORE_SIGMOID, n_group, topk_group, group_top, E / n_group,
                    renorm ? 1 : 0, route_scale, topk_ids, topk_weights};
  if (E <= 64) launch_fw<1>(a, stream);
  else if (E <= 128) launch_fw<2>(a, stream);
  else if (E <= 256) launch_fw<4>(a, stream);
  else if (E <= 512) launch_fw<8>(a, stream);
  else launch_fw<16>(a, stream);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

extern "C" moe_status moe_router_group_topk_backward(const float* logits, const int32_t* topk_ids,
                                                     const float* d_weights, int T, int E, int K, moe_score score,
                                                     int renorm, float route_scale, float* d_logits,
                                                     hipStream_t stream) {
  MOE_CHECK(T >= 0 && E >= 1 && K >= 1 && K <= E, MOE_ERR_INVALID_ARG);
  MOE_CHECK(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID, MOE_ERR_INVALID_ARG);
  MOE_CHECK(E <= kMaxE && K <= kMaxK, MOE_ERR_UNSUPPORTED);
  MOE_CHECK(route_scale == route_scale && fabsf(route_scale) < INFINITY, MOE_ERR_INVALID_ARG);
  if (T == 0) return MOE_OK;
  MOE_CHECK(logits && topk_ids && d_weights && d_logits && d_logits != logits, MOE_ERR_INVALID_ARG);
  RouteArgs a{};
  a.logits = logits;
  a.T = T;
  a.E = E;
  a.K = K;
  a.sigmoid = score == MOE_SCORE_SIGMOID;
  a.renorm = renorm ? 1 : 0;
  a.scale = route_scale;
  a.ids = const_cast<int32_t*>(topk_ids);
  if (E <= 64) launch_bw<1>(a, d_weights, d_logits, stream);
  else if (E <= 128) launch_bw<2>(a, d_weights, d_logits, stream);
  else if (E <= 256) launch_bw<4>(a, d_weights, d_logits, stream);
  else if (E <= 512) launch_bw<8>(a, d_weights, d_logits, stream);
  else launch_bw<16>(a, d_weights, d_logits, stream);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}
