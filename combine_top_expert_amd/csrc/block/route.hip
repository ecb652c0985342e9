// moe_router_group_topk and its backward.
//
// One wavefront per token; lane l holds the NPL neighbours l NPL, l NPL + 1, ...
// so a row is read with one wide load per lane and a group of experts is
// usually a run of lanes, whose two best scores meet in a few DPP steps.  A
// score c = s + bias is held as the order-preserving 32-bit key of the router's
// top-K (NaN lowest among the live, 0 for a masked or retired entry).  Every
// lane sorts its keys once; a selection round is then a wave maximum of the
// lanes' heads, a ballot for the lowest lane that holds it, and a shift of that
// lane's list.  Lanes are in expert order and the sort is stable, so equal keys
// go to the lower id.
//
// The order is the one of exact scores.  Without a bias it is the logits' order,
// which needs no arithmetic.  Where arithmetic decides (a bias, or the sums that
// rank the groups), an fp32 score is off by at most a few 2^-24 of the row's
// scores; a row in which two neighbours of the order lie within that of each
// other is decided again by the same wave in fp64 (route_exact).

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
constexpr float kU = 5.9604644775390625e-8f;   // 2^-24, half a step of fp32

struct RouteArgs {
  const float* logits;
  const float* bias;
  int T, E, K;
  int sigmoid;
  int n_group, topk_group, group_top, group_size;
  int renorm;
  float scale;
  int vec;                      // rows may be read NPL logits at a time
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

// exp(d) by the hardware's exp2: within (1.1 |d| + 2) kU of itself
__device__ __forceinline__ float fast_exp(float d) { return __builtin_amdgcn_exp2f(d * 1.44269504088896341f); }

// Sorts K[0..N) descending, I along with it (odd-even transposition for two,
// else a merge network); keys of equal value keep their order.
template <int N> __device__ __forceinline__ void sort_desc(uint32_t (&k)[N], int (&id)[N]) {
  // stable: an exchange only where the later key is strictly larger, between
  // neighbours; N is small and the network unrolled
#pragma unroll
  for (int pass = 0; pass < N; ++pass)
#pragma unroll
    for (int i = pass & 1; i + 1 < N; i += 2) {
      const bool sw = k[i + 1] > k[i];
      const uint32_t hi = max(k[i], k[i + 1]), lo = min(k[i], k[i + 1]);
      const int a = sw ? id[i + 1] : id[i], b = sw ? id[i] : id[i + 1];
      k[i] = hi; k[i + 1] = lo;
      id[i] = a; id[i + 1] = b;
    }
}

// (t1, t2) <- the two largest of this lane's and its partner's
template <int CTRL> __device__ __forceinline__ void merge2(uint32_t& t1, uint32_t& t2) {
  const uint32_t o1 = moe_router::dpp_u32<CTRL>(t1, t1), o2 = moe_router::dpp_u32<CTRL>(t2, t2);
  t2 = max(min(t1, o1), max(t2, o2));
  t1 = max(t1, o1);
}
__device__ __forceinline__ void merge2_shfl(uint32_t& t1, uint32_t& t2, int d) {
  const uint32_t o1 = __shfl_xor(t1, d), o2 = __shfl_xor(t2, d);
  t2 = max(min(t1, o1), max(t2, o2));
  t1 = max(t1, o1);
}

template <int NPL>   // scores per lane: E <= 64 * NPL
__global__ __launch_bounds__(kThreads) void group_topk_kernel(RouteArgs a) {
  extern __shared__ double lds[];
  const int lane = moe::lane_id();
  const int wave = threadIdx.x >> 6;
  const int t = blockIdx.x * kWaves + wave;
  if (t >= a.T) return;
  const float* row = a.logits + static_cast<int64_t>(t) * a.E;
  const int e0 = lane * NPL;

  float l[NPL], b[NPL];
  if (NPL > 1 && a.vec) {
    typedef float vec_t __attribute__((ext_vector_type(NPL < 4 ? NPL : 4)));
    constexpr int W = NPL < 4 ? NPL : 4;
#pragma unroll
    for (int j = 0; j < NPL; j += W) {
      vec_t v = {}, w = {};
      if (e0 < a.E) {
        v = *reinterpret_cast<const vec_t*>(row + e0 + j);
        if (a.bias) w = *reinterpret_cast<const vec_t*>(a.bias + e0 + j);
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        l[j + i] = e0 < a.E ? v[i] : -INFINITY;
        b[j + i] = w[i];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      l[j] = e0 + j < a.E ? row[e0 + j] : -INFINITY;
      b[j] = a.bias && e0 + j < a.E ? a.bias[e0 + j] : 0.f;
    }
  }

  float m = 0.f, sum = 1.f, inv = 1.f;
  if (!a.sigmoid) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (!(l[j] <= kMask)) m = fmaxf(m, l[j]);
    m = wave_max_f32(m);
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (!(l[j] <= kMask)) sum += fast_exp(l[j] - m);
    sum = wave_sum_f32(sum);
    inv = 1.0f / sum;
  }
  auto fast_score = [&](float x) {
    return a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + fast_exp(-x)) : fast_exp(x - m) * inv;
  };

  // Keys: of the logits without a bias, of c with one.  fast_score is off by at
  // most (1.1 |d| + 2 + 1 + 2) kU of itself (d: the exponent; exp, add and
  // reciprocal), for softmax by the sum's and the quotient's roundings too
  // (NPL + 6 additions, terms that are off by 5 kU on average at most).
  const float c0 = a.sigmoid ? 6.f : 20.f + NPL;
  uint32_t key[NPL];
  int id[NPL];
  float err = 0.f;
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    key[j] = 0;
    id[j] = e0 + j;
    const bool live = !(l[j] <= kMask);
    if (a.bias) {
      const float s = fast_score(l[j]), v = s + b[j];
      if (live && !(b[j] <= kMask)) {
        key[j] = max(score_key(v), 1u);
        const float d = a.sigmoid ? l[j] : l[j] - m;
        err = fmaxf(err, fmaf(s, fmaf(1.5f, fabsf(d), c0), fabsf(v) < INFINITY ? fabsf(v) : 0.f));
      }
    } else if (live) {
      key[j] = sum != sum ? 1u : max(score_key(l[j]), 1u);
    }
  }
  // how far a c may be off: 0 without a bias, where keys are exact
  const float tol = a.bias ? wave_max_f32(err) * kU : 0.f;

  bool near = false;
  if (a.n_group > 1) {
    const int gs = a.group_size;
    const int lg = gs / NPL;                            // lanes of a group
    const bool runs = gs % NPL == 0 && (lg & (lg - 1)) == 0;
    uint32_t t1 = 0, t2 = 0;
    int g, stride;                                      // this lane's group, lanes between groups
    if (runs) {
#pragma unroll
      for (int j = 0; j < NPL; ++j) {
        t2 = max(t2, min(t1, key[j]));
        t1 = max(t1, key[j]);
      }
      if (lg >= 2) merge2<moe_router::kDppXor1>(t1, t2);
      if (lg >= 4) merge2<moe_router::kDppXor2>(t1, t2);
      if (lg >= 8) merge2<moe_router::kDppHalfMirror>(t1, t2);
      if (lg >= 16) merge2<moe_router::kDppMirror>(t1, t2);
      if (lg >= 32) merge2_shfl(t1, t2, 16);
      if (lg >= 64) merge2_shfl(t1, t2, 32);
      g = lane >> __builtin_ctz(lg);
      stride = lg;
    } else {
      uint32_t* c32 = reinterpret_cast<uint32_t*>(lds + static_cast<size_t>(wave) * a.E);
#pragma unroll
      for (int j = 0; j < NPL; ++j)
        if (e0 + j < a.E) c32[e0 + j] = key[j];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (lane < a.n_group)
        for (int i = 0; i < gs; ++i) {
          const uint32_t k = c32[lane * gs + i];
          t2 = max(t2, min(t1, k));
          t1 = max(t1, k);
        }
      g = lane;
      stride = 1;
    }
    // the group's score; dead groups keep key 0
    uint32_t gkey = 0;
    if (t1 && g < a.n_group) {
      float v = key_value(t1);
      if (a.group_top == 2) {
        if (!a.bias) v = fast_score(v);
        if (t2) v += a.bias ? key_value(t2) : fast_score(key_value(t2));
      }
      gkey = max(score_key(v), 1u);
    }
    int rank = 0;
    for (int h = 0; h < a.n_group; ++h) {
      const uint32_t o = __builtin_amdgcn_readlane(gkey, h * stride);
      rank += (o > gkey || (o == gkey && h < g)) ? 1 : 0;
    }
    const bool kept = g < a.n_group && rank < a.topk_group;
    // the last group that stays and the first that does not
    const uint64_t in = __ballot(g < a.n_group && rank == a.topk_group - 1);
    const uint64_t out = __ballot(g < a.n_group && rank == a.topk_group);
    if (out && (a.bias || a.group_top == 2)) {
      const uint32_t ki = __builtin_amdgcn_readlane(gkey, __builtin_ctzll(in));
      const uint32_t ko = __builtin_amdgcn_readlane(gkey, __builtin_ctzll(out));
      if (ki > 1 && ko > 1) {
        const float vi = key_value(ki), vo = key_value(ko);
        // without a bias a sum of two scores is off by its own share
        // (exponents to 88) and by what fp32 loses below its normal range
        near = vi - vo <= (a.bias ? 4.f * tol + 2.f * kU * (fabsf(vi) + fabsf(vo)) : (c0 + 140.f) * kU * (vi + vo) + 1e-37f);
      }
    }
    if (runs) {
#pragma unroll
      for (int j = 0; j < NPL; ++j) key[j] = kept ? key[j] : 0u;
    } else {
      const uint64_t keep = __ballot(kept);
#pragma unroll
      for (int j = 0; j < NPL; ++j)
        if (e0 + j < a.E && !((keep >> ((e0 + j) / gs)) & 1)) key[j] = 0;
    }
  }

  int my = -1;
  if (!near) {
    sort_desc<NPL>(key, id);
    uint32_t mine = 0;                                  // lane k: round k's key, lane K: the runner-up's
    for (int k = 0; k <= a.K; ++k) {
      const uint32_t win = wave_max_u32(key[0]);
      if (win == 0) break;
      const int owner = __builtin_ctzll(__ballot(key[0] == win));
      if (lane == k) mine = win;
      const int e = __builtin_amdgcn_readlane(id[0], owner);
      if (lane == k) my = e;
      if (lane == owner) {
#pragma unroll
        for (int j = 0; j + 1 < NPL; ++j) {
          key[j] = key[j + 1];
          id[j] = id[j + 1];
        }
        key[NPL - 1] = 0;
      }
    }
    if (a.bias) {
      const uint32_t next = __shfl_down(mine, 1);
      near = __ballot(lane < a.K && mine > 1 && next > 1 && key_value(mine) - key_value(next) <= 2.f * tol) != 0;
    }
  }
  if (near) my = route_exact(a, row, lds + static_cast<size_t>(wave) * a.E, lane);

  // lane k's logit, from the lane that holds it
  float x = 0.f;
  if constexpr (NPL <= 4) {
    const int from = max(my, 0) / NPL;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      const float v = __shfl(l[j], from);
      x = max(my, 0) % NPL == j ? v : x;
    }
  } else {
    x = row[max(my, 0)];
  }
  const bool real = lane < a.K && my >= 0;
  float w = real ? (a.sigmoid ? sigmoid_f(x) : expf(x - m) / sum) : 0.f;
  if (a.renorm) w = w / (wave_sum_f32(w) + 1e-20f);
  if (lane < a.K) {
    a.ids[static_cast<int64_t>(t) * a.K + lane] = my;
    a.weights[static_cast<int64_t>(t) * a.K + lane] = real ? w * a.scale : 0.f;
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

template <int NPL> void launch_fw(RouteArgs a, hipStream_t stream) {
  const int grid = (a.T + kWaves - 1) / kWaves;
  a.vec = a.E % NPL == 0 && aligned16(a.logits) && aligned16(a.bias);
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
                    renorm ? 1 : 0, route_scale, 0, topk_ids, topk_weights};
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
