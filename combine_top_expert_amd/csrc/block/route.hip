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
// The order is the one of fp64 scores.  Without a bias it is the logits' order,
// which needs no arithmetic, as long as fp64 tells the scores apart (may_tie).
// Where arithmetic decides (a bias, or the sums that rank the groups), an fp32
// score is off by at most a few 2^-24 of the row's scores.  A row in which two
// neighbours of the order may tie, or lie within that of each other, is decided
// again by the same wave in fp64 (route_exact).
//
// Bound by vector instructions: 630 a token in a first form with the same
// layout, 239 in the one for large batches, which takes 31 us for 65536 x 256
// with 4 or all of 8 groups and K = 8 (71 MB, 11 us of memory time).  The fp64 path
// is the other part: an earlier build took 38.6 us with it and 22.4 us without.
// One token a wave, 65536 tokens without a bias, us: 64 experts softmax top-6 24, 128
// softmax top-8 31, 128 sigmoid, 4 of 8 groups by their two best 40, 256 by their
// best 42; 16384 tokens: 384 experts sigmoid with a bias top-8 21, 1024 softmax
// top-32 57.

#include <type_traits>

#include "block_common.h"
#include "router_common.h"

namespace {

using namespace moe_block;
using moe_router::score_key;
using moe_router::wave_max_f32;
using moe_router::wave_sum_f32;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / MOE_WAVE;
constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr float kMask = -3.3e38f;   // covers -inf and the lowest finite fp32 and bf16
constexpr float kU = 5.9604644775390625e-8f;   // 2^-24, half a step of fp32
// An exponential or reciprocal below 2^-126 = 1.2e-38 is flushed to 0, which a
// relative error does not cover: eight of those.
constexpr float kFlush = 1e-37f;

// f(0), f(1), ... f(N - 1) with constant arguments: arrays indexed so stay in
// single registers (a loop that is unrolled later makes the compiler hold
// them as one wide register tuple, copied whole: 256 VGPRs instead of 90 for
// sixteen scores a lane).
template <int N, int I = 0, typename F> __device__ __forceinline__ void each(const F& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}

// e / size for 0 <= e < 1024, inv = 1 / size: (e + 1/2) / size is at least
// 1 / 2048 away from every whole number, far more than its rounding.
__device__ __forceinline__ int group_of(int e, float inv) { return static_cast<int>((static_cast<float>(e) + 0.5f) * inv); }

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

// The wave maximum of keys.  Lanes that a step does not reach read 0, the
// maximum's identity, so that each step is one instruction (the exchange is an
// operand modifier of the maximum).
template <int CTRL, int ROWS = 0xF> __device__ __forceinline__ uint32_t max_step(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xF, true)));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max_step<moe_router::kDppXor1>(v);
  v = max_step<moe_router::kDppXor2>(v);
  v = max_step<moe_router::kDppHalfMirror>(v);
  v = max_step<moe_router::kDppMirror>(v);
  v = max_step<moe_router::kDppBcast15, 0xA>(v);
  v = max_step<moe_router::kDppBcast31, 0xC>(v);
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

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

// Order-preserving image of a double: every NaN is 1, below all numbers, -0 and
// +0 map together; 0 stands for a masked or retired entry.
__device__ __forceinline__ uint64_t key64(double v) {
  if (v != v) return 1ull;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key64_value(uint64_t k) {
  if (k <= 1ull) return k ? NAN : -INFINITY;
  return __longlong_as_double(static_cast<int64_t>((k >> 63) ? (k ^ 0x8000000000000000ull) : ~k));
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t k) {
  const uint32_t hi = wave_max_u32(static_cast<uint32_t>(k >> 32));
  const uint32_t lo = wave_max_u32(static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

// The choice in fp64: lane k returns round k's expert, or -1.  Lane l holds
// experts l NPL + j; `lds` is the wave's row of E keys.  Rows come here seldom,
// but a launch ends with its last wave, so this is kept short: selection on
// registers, and every group scanned by as many lanes as there are for it.
template <int NPL, bool SIG, bool BIAS>
__device__ __forceinline__ int route_exact(const RouteArgs& a, const float* __restrict__ row, uint64_t* lds, int lane) {
  const int e0 = lane * NPL;
  float l[NPL];
  double m = -INFINITY, sum = 0.0;
  each<NPL>([&](auto j) {
    l[j] = e0 + j < a.E ? row[e0 + j] : -INFINITY;
  });
  if (!SIG) {
    each<NPL>([&](auto j) {
      if (!(l[j] <= kMask)) m = fmax(m, static_cast<double>(l[j]));
    });
    m = wave_max_f64(m);
    each<NPL>([&](auto j) {
      if (!(l[j] <= kMask)) sum += exp(static_cast<double>(l[j]) - m);
      __builtin_amdgcn_sched_barrier(0);
    });
    sum = wave_sum_f64(sum);
  }
  uint64_t key[NPL];
  each<NPL>([&](auto j) {
    key[j] = 0;
    __builtin_amdgcn_sched_barrier(0);      // one fp64 exponential's registers at a time
    if (l[j] <= kMask) return;
    double v = SIG ? 1.0 / (1.0 + exp(-static_cast<double>(l[j]))) : exp(static_cast<double>(l[j]) - m) / sum;
    if (BIAS) {
      if (a.bias[e0 + j] <= kMask) return;
      v += static_cast<double>(a.bias[e0 + j]);
    }
    key[j] = key64(v);
  });
  if (a.n_group > 1) {
    each<NPL>([&](auto j) {
      if (e0 + j < a.E) lds[e0 + j] = key[j];
    });
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int shift = 31 - __builtin_clz(MOE_WAVE / a.n_group), P = 1 << shift;   // lanes that scan a group
    const int g = lane >> shift;
    uint64_t t1 = 0, t2 = 0;
    if (g < a.n_group)
      for (int i = lane & (P - 1); i < a.group_size; i += P) {
        const uint64_t k = lds[g * a.group_size + i];
        t2 = max(t2, min(t1, k));
        t1 = max(t1, k);
      }
    for (int d = 1; d < P; d <<= 1) {
      const uint64_t o1 = __shfl_xor(t1, d), o2 = __shfl_xor(t2, d);
      t2 = max(min(t1, o1), max(t2, o2));
      t1 = max(t1, o1);
    }
    uint64_t gk = 0;
    if (t1) gk = (a.group_top == 2 && t2) ? key64(key64_value(t1) + key64_value(t2)) : t1;
    int rank = 0;
    for (int h = 0; h < a.n_group; ++h) {
      const uint64_t o = __shfl(gk, h << shift);
      rank += (o > gk || (o == gk && h < g)) ? 1 : 0;
    }
    const uint64_t keep = __ballot(g < a.n_group && rank < a.topk_group);
    const float inv = 1.0f / static_cast<float>(a.group_size);
    each<NPL>([&](auto j) {
      if (e0 + j < a.E && !((keep >> (group_of(e0 + j, inv) << shift)) & 1)) key[j] = 0;
    });
  }
  int my = -1;
#pragma unroll 1
  for (int k = 0; k < a.K; ++k) {
    uint64_t best = 0;
    int be = 0;
    each<NPL>([&](auto j) {
      if (key[j] > best) {
        best = key[j];
        be = e0 + j;
      }
    });
    const uint64_t win = wave_max_u64(best);
    if (win == 0) break;
    const int e = __builtin_amdgcn_readlane(be, __builtin_ctzll(__ballot(best == win)));
    each<NPL>([&](auto j) {
      if (e0 + j == e) key[j] = 0;
    });
    if (lane == k) my = e;
  }
  return my;
}

// exp(d) by the hardware's exp2: within (1.1 |d| + 2) kU of itself
__device__ __forceinline__ float fast_exp(float d) { return __builtin_amdgcn_exp2f(d * 1.44269504088896341f); }

// Sorts k descending, id along with it, by N passes of exchanges between
// neighbours where the later key is strictly larger: equal keys keep their
// order.  (Recursion, so that every index is a constant.)
template <int PASS, int I, int N> __device__ __forceinline__ void stable_sort(uint32_t (&k)[N], int (&id)[N]) {
  if constexpr (PASS < N) {
    if constexpr (I + 1 < N) {
      const bool sw = k[I + 1] > k[I];
      const uint32_t hi = max(k[I], k[I + 1]), lo = min(k[I], k[I + 1]);
      const int a = sw ? id[I + 1] : id[I], b = sw ? id[I] : id[I + 1];
      k[I] = hi; k[I + 1] = lo;
      id[I] = a; id[I + 1] = b;
      stable_sort<PASS, I + 2>(k, id);
    } else {
      stable_sort<PASS + 1, (PASS + 1) & 1>(k, id);
    }
  }
}

// (t1, t2) <- the two largest of this lane's and its partner's
template <int CTRL> __device__ __forceinline__ void merge2(uint32_t& t1, uint32_t& t2) {
  const uint32_t o1 = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(t1), CTRL, 0xF, 0xF, true));
  t2 = max(min(t1, o1), max_step<CTRL>(t2));
  t1 = max(t1, o1);
}
__device__ __forceinline__ void merge2_shfl(uint32_t& t1, uint32_t& t2, int d) {
  const uint32_t o1 = __shfl_xor(t1, d), o2 = __shfl_xor(t2, d);
  t2 = max(min(t1, o1), max(t2, o2));
  t1 = max(t1, o1);
}

template <int NPL, bool SIG, bool BIAS>   // scores per lane: E <= 64 * NPL
__global__ __launch_bounds__(kThreads) void group_topk_kernel(RouteArgs a) {
  extern __shared__ uint64_t lds[];
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
        if (BIAS) w = *reinterpret_cast<const vec_t*>(a.bias + e0 + j);
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        l[j + i] = e0 < a.E ? v[i] : -INFINITY;
        b[j + i] = w[i];
      }
    }
  } else {
    each<NPL>([&](auto j) {
      l[j] = e0 + j < a.E ? row[e0 + j] : -INFINITY;
      b[j] = BIAS && e0 + j < a.E ? a.bias[e0 + j] : 0.f;
    });
  }

  float m = 0.f, sum = 1.f, inv = 1.f;
  if (!SIG) {
    m = -INFINITY;
    each<NPL>([&](auto j) {
      if (!(l[j] <= kMask)) m = fmaxf(m, l[j]);
    });
    m = wave_max_f32(m);
    sum = 0.f;
    each<NPL>([&](auto j) {
      if (!(l[j] <= kMask)) sum += fast_exp(l[j] - m);
    });
    sum = wave_sum_f32(sum);
    inv = 1.0f / sum;
  }
  auto fast_score = [&](float x) {
    return SIG ? __builtin_amdgcn_rcpf(1.0f + fast_exp(-x)) : fast_exp(x - m) * inv;
  };

  // Keys: of the logits without a bias, of c with one.  fast_score is off by at
  // most (1.1 |d| + 2 + 1 + 2) kU of itself (d: the exponent; exp, add and
  // reciprocal), for softmax by the sum's and the quotient's roundings too
  // (NPL + 6 additions, terms that are off by 5 kU on average at most).
  const float c0 = SIG ? 6.f : 20.f + NPL;

  // Whether logits v > o may have the same fp64 score.  Neighbouring fp32 logits
  // have different ones, but for sigmoid from 23 on, where 1 + exp(-l) is rounded
  // to steps of 2^-52 (from 37 on all are 1; fast_exp is off by 3e-15 at 20, less
  // above), where the score underflows (-708 below the largest, with sigmoid below
  // 0), and next to 0, where logits lie closer than fp64 can tell 1 + l (or l less
  // the largest) apart.
  auto may_tie = [&](float v, float o) {
    const bool out = SIG ? (o > 20.f && fast_exp(-o) - fast_exp(-v) < 8e-15f) || v < -700.f : v - m < -700.f;
    return v > o && (v - o < 1e-12f || out);
  };
  // whether it can hold at all: of two logits, both below 2^-15 (1e-12 apart
  // means that), or outside an ordinary range
  auto two_in_zone = [&](bool live, float v) {
    const bool in = fabsf(v) < 0x1p-15f || (SIG ? fabsf(v) > 20.f : v - m < -700.f);
    return __popcll(__ballot(live && in)) > 1;
  };
  uint32_t key[NPL];
  int id[NPL];
  float err = 0.f, all = 0.f;
  each<NPL>([&](auto j) {
    id[j] = e0 + j;
    asm("" : "+v"(id[j]));            // a value to move along, not an index to select by
    if (BIAS) {
      // plain order-preserving image: -0 below +0 and NaN anywhere, but equal
      // scores and NaN are decided in fp64 below
      const float s = fast_score(l[j]), v = s + b[j];
      const uint32_t u = __float_as_uint(v);
      const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
      const bool live = !(l[j] <= kMask) && !(b[j] <= kMask);
      const float d = SIG ? l[j] : l[j] - m;
      key[j] = live ? k : 0u;
      err = fmaxf(err, live ? fmaf(s, fmaf(1.5f, fabsf(d), c0), fabsf(v)) : 0.f);
      all += live ? v : 0.f;
    } else {
      key[j] = l[j] <= kMask ? 0u : (sum != sum ? 1u : max(score_key(l[j]), 1u));
    }
  });
  // how far a c may be off: 0 without a bias, where keys are exact
  const float tol = BIAS ? wave_max_f32(err) * kU + kFlush : 0.f;

  bool near = BIAS && __ballot(all != all) != 0;       // a NaN among the scores
  if (a.n_group > 1 && !near) {
    const int gs = a.group_size;
    const int lg = gs / NPL;                            // lanes of a group
    const bool runs = gs % NPL == 0 && (lg & (lg - 1)) == 0;
    uint32_t t1 = 0, t2 = 0;
    int g, stride;                                      // this lane's group, lanes between groups
    if (runs) {
      each<NPL>([&](auto j) {
        t2 = max(t2, min(t1, key[j]));
        t1 = max(t1, key[j]);
      });
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
      each<NPL>([&](auto j) {
        if (e0 + j < a.E) c32[e0 + j] = key[j];
      });
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
    bool look = true;                                   // at the edge between the groups that stay and the others
    if (!BIAS && a.group_top == 1) {
      gkey = g < a.n_group ? t1 : 0u;
      look = two_in_zone(gkey > 1, key_value(gkey));
    } else if (t1 && g < a.n_group) {
      float v = key_value(t1);
      if (a.group_top == 2) {
        if (!BIAS) v = fast_score(v);
        if (t2) v += BIAS ? key_value(t2) : fast_score(key_value(t2));
      }
      gkey = max(score_key(v), 1u);
    }
    int rank = 0;
    for (int h = 0; h < a.n_group; ++h) {
      // o > gkey, or o == gkey from a lower group
      const uint32_t o = __builtin_amdgcn_readlane(gkey, h * stride);
      rank += o + (h < g ? 1u : 0u) > gkey ? 1 : 0;
    }
    const bool kept = g < a.n_group && rank < a.topk_group;
    // the last group that stays and the first that does not
    const uint64_t in = __ballot(g < a.n_group && rank == a.topk_group - 1);
    const uint64_t out = __ballot(g < a.n_group && rank == a.topk_group);
    if (out && look) {
      const uint32_t ki = __builtin_amdgcn_readlane(gkey, __builtin_ctzll(in));
      const uint32_t ko = __builtin_amdgcn_readlane(gkey, __builtin_ctzll(out));
      if (ki > 1 && ko > 1) {
        const float vi = key_value(ki), vo = key_value(ko);
        // without a bias a sum of two scores is off by its own share
        // (exponents to 88) and by what fp32 loses below its normal range
        near = BIAS ? vi - vo <= 4.f * tol + 2.f * kU * (fabsf(vi) + fabsf(vo))
               : a.group_top == 2 ? vi - vo <= (c0 + 140.f) * kU * (vi + vo) + kFlush : may_tie(vi, vo);
      }
    }
    if (runs) {
      each<NPL>([&](auto j) {
        key[j] = kept ? key[j] : 0u;
      });
    } else {
      const uint64_t keep = __ballot(kept);
      each<NPL>([&](auto j) {
        if (e0 + j < a.E && !((keep >> group_of(e0 + j, 1.0f / static_cast<float>(gs))) & 1)) key[j] = 0;
      });
    }
  }

  int my = -1;
  if (!near) {
    stable_sort<0, 0>(key, id);
    uint32_t mine = 0;                                  // lane k: round k's key, lane K: the runner-up's
    for (int k = 0; k <= a.K; ++k) {
      const uint32_t win = wave_max_u32(key[0]);
      if (win == 0) break;
      const int owner = __builtin_ctzll(__ballot(key[0] == win));
      const int e = __builtin_amdgcn_readlane(id[0], owner);
      mine = lane == k ? win : mine;
      my = lane == k ? e : my;
      if (lane == owner) {
        each<NPL - 1>([&](auto j) {
          key[j] = key[j + 1];
          id[j] = id[j + 1];
        });
        key[NPL - 1] = 0;
      }
    }
    if (BIAS) {
      const uint32_t next = __shfl_down(mine, 1);
      near = __ballot(lane < a.K && mine > 1 && next > 1 && key_value(mine) - key_value(next) <= 2.f * tol) != 0;
    }
  }

  // lane k's logit, from the lane that holds it (lane K: the runner-up's)
  auto logit = [&]() {
    float v = 0.f;
    if constexpr (NPL <= 4) {
      const int from = max(my, 0) / NPL;
      each<NPL>([&](auto j) {
        const float o = __shfl(l[j], from);
        v = max(my, 0) % NPL == j ? o : v;
      });
    } else {
      v = row[max(my, 0)];
    }
    return v;
  };
  float x = logit();
  if (!BIAS && !near) {
    if (two_in_zone(my >= 0, x)) {
      const float o = __shfl_down(x, 1);
      const int next = __shfl_down(my, 1);              // by every lane: lane K - 1 reads lane K
      near = __ballot(lane < a.K && next >= 0 && may_tie(x, o)) != 0;
    }
  }
  if (near) {
    my = route_exact<NPL, SIG, BIAS>(a, row, lds + static_cast<size_t>(wave) * a.E, lane);
    x = logit();
  }
  const bool real = lane < a.K && my >= 0;
  float w = real ? (SIG ? sigmoid_f(x) : expf(x - m) / sum) : 0.f;
  if (a.renorm) w = w / (wave_sum_f32(w) + 1e-20f);
  if (lane < a.K) {
    a.ids[static_cast<int64_t>(t) * a.K + lane] = my;
    a.weights[static_cast<int64_t>(t) * a.K + lane] = real ? w * a.scale : 0.f;
  }
}

// Four tokens per wave, one per 16-lane row of lanes, for large batches with a
// bias: everything stays in the row (a row maximum is four DPP steps and all
// lanes have it), and one instruction works for four tokens.  A lane holds NPL
// (8 or 16) neighbouring experts.
//
// Keys are the order-preserving images of c with the four lowest bits replaced
// by 15 - j, j the expert's place in its lane, so that sorting moves one
// register per expert; what the truncation hides (32 kU of c) is added to the
// distance below which a row is decided in fp64.  At most kSegK experts are
// taken, so a lane's list is kept to its kSegK + 1 largest.
constexpr int kSeg = 16;
constexpr int kSegK = 8;

// Sorts k[LO .. LO + N) descending by Batcher's odd-even merges (63 exchanges
// of 16 keys).
template <int A, int B, int M> __device__ __forceinline__ void exchange(uint32_t (&k)[M]) {
  const uint32_t hi = max(k[A], k[B]);
  k[B] = min(k[A], k[B]);
  k[A] = hi;
}
template <int LO, int N, int R, int I, int M> __device__ __forceinline__ void merge_odd(uint32_t (&k)[M]) {
  if constexpr (I + R < LO + N) {
    exchange<I, I + R>(k);
    merge_odd<LO, N, R, I + 2 * R>(k);
  }
}
template <int LO, int N, int R, int M> __device__ __forceinline__ void merge_sorted(uint32_t (&k)[M]) {
  if constexpr (2 * R < N) {
    merge_sorted<LO, N, 2 * R>(k);
    merge_sorted<LO + R, N, 2 * R>(k);
    merge_odd<LO, N, R, LO + R>(k);
  } else {
    exchange<LO, LO + R>(k);
  }
}
template <int LO, int N, int M> __device__ __forceinline__ void merge_sort_desc(uint32_t (&k)[M]) {
  if constexpr (N > 1) {
    merge_sort_desc<LO, N / 2>(k);
    merge_sort_desc<LO + N / 2, N / 2>(k);
    merge_sorted<LO, N, 1>(k);
  }
}

// the lowest set bit of each 16-bit field
__device__ __forceinline__ uint64_t lowest_of_rows(uint64_t m) {
  constexpr uint64_t top = 0x8000800080008000ull, one = 0x0001000100010001ull;
  const uint64_t n = ~m;
  return m & (((n & ~top) + one) ^ (n & top));          // m & -m, field by field
}

template <int CTRL> __device__ __forceinline__ void merge2f(float& t1, float& t2) {
  const float o1 = moe_router::dpp_f32<CTRL>(t1, t1), o2 = moe_router::dpp_f32<CTRL>(t2, t2);
  t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
  t1 = fmaxf(t1, o1);
}

template <int NPL, bool SIG>
__global__ __launch_bounds__(kThreads) void group_topk_seg_kernel(RouteArgs a) {
  extern __shared__ uint64_t lds[];
  __shared__ uint2 ring[kWaves][MOE_WAVE / kSeg][kSegK + 1];
  const int lane = moe::lane_id();
  const int wave = threadIdx.x >> 6;
  const int sl = lane & (kSeg - 1), seg = lane / kSeg;
  const int t0 = (blockIdx.x * kWaves + wave) * (MOE_WAVE / kSeg);
  if (t0 >= a.T) return;
  const int t = min(t0 + seg, a.T - 1);                 // a row past the end repeats the last, unstored
  const float* row = a.logits + static_cast<int64_t>(t) * a.E;
  const int e0 = sl * NPL;
  const bool used = e0 < a.E;

  float l[NPL], c[NPL];
#pragma unroll
  for (int j = 0; j < NPL; j += 4) {
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY), w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (used) {
      v = *reinterpret_cast<const float4*>(row + e0 + j);
      w = *reinterpret_cast<const float4*>(a.bias + e0 + j);
    }
    l[j] = v.x; l[j + 1] = v.y; l[j + 2] = v.z; l[j + 3] = v.w;
    c[j] = w.x; c[j + 1] = w.y; c[j + 2] = w.z; c[j + 3] = w.w;
  }
  float lmax = -INFINITY;
  each<NPL>([&](auto j) {
    lmax = fmaxf(lmax, l[j]);
  });
  lmax = moe_router::row_max_f32(lmax);
  float sum = 1.f, inv = 1.f;
  if (!SIG) {
    sum = 0.f;
    each<NPL>([&](auto j) {
      sum += l[j] <= kMask ? 0.f : fast_exp(l[j] - lmax);
    });
    sum = moe_router::row_sum_f32(sum);
    inv = 1.0f / sum;
  }
  // c, and the rows whose scores are no ordinary numbers
  uint64_t odd = 0;
  each<NPL>([&](auto j) {
    const float s = SIG ? __builtin_amdgcn_rcpf(1.0f + fast_exp(-l[j])) : fast_exp(l[j] - lmax) * inv;
    c[j] = l[j] <= kMask ? -INFINITY : s + c[j];
    odd |= __ballot(!(c[j] < INFINITY));
  });
  bool near = ((odd >> (seg * kSeg)) & 0xffffu) != 0;
  // How far a c may be off, its own rounding aside: fast_exp's share of s grows
  // with the exponent, but s |l| is at most smax |lmax| + 1.3 smax (sigmoid), and
  // exp(-d) d at most 0.37 (softmax, plus the sum's NPL + 4 additions).  |lmax| is
  // cut where sigmoid is 0 or 1 to fp32: far below, smax is 0 and the product has
  // to stay a number.
  const float smax = SIG ? __builtin_amdgcn_rcpf(1.0f + fast_exp(-lmax)) : inv;
  const float tol = smax * (SIG ? 8.f + 1.5f * fminf(fabsf(lmax), 128.f) : 20.f + NPL) * kU + kFlush;

  bool kept = true;
  if (a.n_group > 1) {
    const int lg = a.group_size / NPL;                  // lanes of a group, a power of two
    float t1 = -INFINITY, t2 = -INFINITY;
    each<NPL>([&](auto j) {
      t2 = __builtin_amdgcn_fmed3f(t1, t2, c[j]);
      t1 = fmaxf(t1, c[j]);
    });
    if (lg >= 2) merge2f<moe_router::kDppXor1>(t1, t2);
    if (lg >= 4) merge2f<moe_router::kDppXor2>(t1, t2);
    if (lg >= 8) merge2f<moe_router::kDppHalfMirror>(t1, t2);
    if (lg >= 16) merge2f<moe_router::kDppMirror>(t1, t2);
    const bool dead = !(t1 > kMask);
    const float gs = dead ? -INFINITY : (a.group_top == 2 && t2 > kMask) ? t1 + t2 : t1;
    int rank = 0;
    for (int h = 0; h < a.n_group; ++h) rank += __shfl(gs, h * lg, kSeg) > gs ? 1 : 0;
    kept = !dead && rank < a.topk_group;
    // the worst group that stays against the best live one that does not, if
    // there is one; equal scores share a rank, so a tie at the edge keeps too many
    const float vi = -moe_router::row_max_f32(kept ? -gs : -INFINITY);
    const float vo = moe_router::row_max_f32(kept ? -INFINITY : gs);
    const uint32_t lanes = static_cast<uint32_t>(__ballot(kept && used) >> (seg * kSeg)) & 0xffffu;
    near |= (vo > -INFINITY && vi - vo <= 4.f * tol + 4.f * kU * (fabsf(vi) + fabsf(vo))) ||
            __popc(lanes) > a.topk_group * lg;
  }

  uint32_t key[NPL];
  each<NPL>([&](auto j) {
    const uint32_t u = __float_as_uint(c[j]);
    const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
    key[j] = ((kept && c[j] > kMask ? k : 0u) & ~15u) | (15u - j);
  });
  merge_sort_desc<0, NPL>(key);
  constexpr int kKeep = NPL < kSegK + 1 ? NPL : kSegK + 1;
  for (int k = 0; k <= a.K; ++k) {
    uint32_t win = max_step<moe_router::kDppXor1>(key[0]);
    win = max_step<moe_router::kDppXor2>(win);
    win = max_step<moe_router::kDppHalfMirror>(win);
    win = max_step<moe_router::kDppMirror>(win);
    const uint64_t owners = lowest_of_rows(__ballot(key[0] == win));
    if ((owners >> lane) & 1) {
      ring[wave][seg][k] = make_uint2(win, e0 + 15 - (win & 15u));
      each<kKeep - 1>([&](auto j) {
        key[j] = key[j + 1];
      });
      key[kKeep - 1] = 0;
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();

  int my = -1;
  if (sl < a.K) {
    const uint2 w = ring[wave][seg][sl], next = ring[wave][seg][sl + 1];
    if (w.x > 15u) {
      my = static_cast<int>(w.y);
      const float v = key_value(w.x & ~15u), o = key_value(next.x & ~15u);
      near |= next.x > 15u && v - o <= 2.f * tol + 40.f * kU * fmaxf(fabsf(v), fabsf(o));
    }
  }
  // the tokens that are decided in fp64, one after the other by the whole wave
  const uint64_t again = __ballot(near);
#pragma unroll 1
  for (int g = 0; g < MOE_WAVE / kSeg; ++g) {
    if (((again >> (g * kSeg)) & 0xffffu) == 0 || t0 + g >= a.T) continue;
    const int id = route_exact<NPL / 4, SIG, true>(a, a.logits + static_cast<int64_t>(t0 + g) * a.E,
                                          lds + static_cast<size_t>(wave) * a.E, lane);
    const int moved = __shfl(id, sl);
    if (seg == g) my = sl < a.K ? moved : -1;
  }

  float w = 0.f;
  if (my >= 0) {
    const float x = row[my];
    w = SIG ? sigmoid_f(x) : expf(x - lmax) / sum;
  }
  if (a.renorm) w = w / (moe_router::row_sum_f32(w) + 1e-20f);
  if (sl < a.K && t0 + seg < a.T) {
    a.ids[static_cast<int64_t>(t) * a.K + sl] = my;
    a.weights[static_cast<int64_t>(t) * a.K + sl] = my >= 0 ? w * a.scale : 0.f;
  }
}

// The sum over this lane's run of SEG (16 or 32) lanes, in every lane of it.
template <int CTRL> __device__ __forceinline__ double dpp_f64(double v) {
  const int64_t u = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xF, 0xF, true);
  return __longlong_as_double(static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo));
}
template <int SEG> __device__ __forceinline__ double seg_sum_f64(double v) {
  v += dpp_f64<moe_router::kDppXor1>(v);
  v += dpp_f64<moe_router::kDppXor2>(v);
  v += dpp_f64<moe_router::kDppHalfMirror>(v);
  v += dpp_f64<moe_router::kDppMirror>(v);
  if constexpr (SEG == 32) v += __shfl_xor(v, 16);
  return v;
}


// a + b where each holds partial sums of its own token in all lanes: afterwards
// the lower half of the lanes (ROW16: of every 32 lanes) holds a's, the upper b's.
template <bool ROW16> __device__ __forceinline__ double halves_f64(double a, double b) {
  const int64_t u = __double_as_longlong(a), v = __double_as_longlong(b);
  auto swap = [](uint32_t x, uint32_t y) {
    if constexpr (ROW16) return __builtin_amdgcn_permlane16_swap(x, y, false, false);
    else return __builtin_amdgcn_permlane32_swap(x, y, false, false);
  };
  const auto lo = swap(static_cast<uint32_t>(u), static_cast<uint32_t>(v));
  const auto hi = swap(static_cast<uint32_t>(u >> 32), static_cast<uint32_t>(v >> 32));
  auto join = [](uint32_t h, uint32_t l) {
    return __longlong_as_double(static_cast<int64_t>((static_cast<uint64_t>(h) << 32) | l));
  };
  return join(hi[0], lo[0]) + join(hi[1], lo[1]);
}

// Whether a rotation of a 16-lane row of v meets `other` in this lane: by 1 to 8,
// which brings every two lanes of the row together once, or by 1 to 15.
template <int SEG, int R = 1> __device__ __forceinline__ bool twice(int v, int other) {
  bool same = other == __builtin_amdgcn_update_dpp(0, v, 0x120 + R, 0xF, 0xF, true);
  if constexpr (R < (SEG == 32 ? 15 : 8)) same |= twice<SEG, R + 1>(v, other);
  return same;
}

// Backward: a wave takes 64 / SEG tokens.  The routes' part is computed for all
// of them at once, route k of token i in lane i SEG + k; then the wave writes
// the rows one after the other: 0 (sigmoid) or the softmax's -s_e dot, and at the
// routes' experts what they computed.  The routes' part is in fp64, an expert
// that occurs twice included: with renormalised weights the terms of ds cancel
// (all of them for K = 1, and the softmax's sum_k ds_k w_k vanishes), and so do
// ds_e and that sum where an expert has nearly all of the softmax.  For that 1 - s
// has to hold, so a row's exponentials, fp32 each, are added in fp64, and a
// route's score is the quotient of the very same two.  With one token a wave the
// routes' part, in which 6 or 8 of 64 lanes work, bound the kernel (8192 x 256,
// K = 8: 6.9 us).
template <int NPL, bool SIG, int SEG>
__global__ __launch_bounds__(kThreads) void group_topk_bw_kernel(RouteArgs a, const float* __restrict__ d_weights,
                                                                 float* __restrict__ d_logits) {
  constexpr int kTok = MOE_WAVE / SEG;
  const int lane = moe::lane_id();
  const int seg = lane / SEG, sl = lane % SEG;
  const int t0 = (blockIdx.x * kWaves + (threadIdx.x >> 6)) * kTok;
  if (t0 >= a.T) return;
  const int e0 = lane * NPL;
  float p[kTok][NPL];                           // the exponentials
  float m = 0.f;                                // of this lane's own token, as what follows
  double inv = 1.0;
  if constexpr (!SIG) {
    each<kTok>([&](auto i) {
      const float* row = a.logits + static_cast<int64_t>(min(t0 + i, a.T - 1)) * a.E;
      each<NPL>([&](auto j) { p[i][j] = e0 + j < a.E ? row[e0 + j] : -INFINITY; });
    });
    double part[kTok];
    each<kTok>([&](auto i) {
      float mi = -INFINITY;
      part[i] = 0.0;
      each<NPL>([&](auto j) { mi = p[i][j] <= kMask ? mi : fmaxf(mi, p[i][j]); });
      mi = wave_max_f32(mi);
      each<NPL>([&](auto j) {
        p[i][j] = p[i][j] <= kMask ? 0.f : expf(p[i][j] - mi);
        part[i] += static_cast<double>(p[i][j]);
      });
      m = seg == i ? mi : m;
    });
    // every token's sum into its own lanes
    double sum;
    if constexpr (kTok == 4) sum = halves_f64<true>(halves_f64<false>(part[0], part[2]), halves_f64<false>(part[1], part[3]));
    else sum = halves_f64<false>(part[0], part[1]);
    sum = seg_sum_f64<SEG>(sum);
    inv = sum == 0.0 ? 0.0 : 1.0 / sum;
  }
  const int t = t0 + seg;
  const bool on = t < a.T && sl < a.K;
  int id = on ? a.ids[static_cast<int64_t>(t) * a.K + sl] : -1;
  if (id >= a.E) id = -1;
  double s = 0.0, d = 0.0, off = 1.0;             // the score, its gradient and, for sigmoid, 1 - s
  if (id >= 0) {
    const float x = a.logits[static_cast<int64_t>(t) * a.E + id];
    if (!(x <= kMask)) {
      if constexpr (SIG) {
        const double e = exp(-fabs(static_cast<double>(x))), r = 1.0 / (1.0 + e);
        s = x < 0.f ? e * r : r;
        off = x < 0.f ? r : e * r;
      } else {
        s = static_cast<double>(expf(x - m)) * inv;
      }
    }
    d = static_cast<double>(d_weights[static_cast<int64_t>(t) * a.K + sl]) * static_cast<double>(a.scale);
  }
  if (a.renorm) {
#pragma clang fp contract(off)
    const double S = seg_sum_f64<SEG>(s) + 1e-20;
    const double mean = seg_sum_f64<SEG>(d * s) / S;
    d = id >= 0 ? (d - mean) / S : 0.0;
  }
  const double dot = SIG ? 0.0 : seg_sum_f64<SEG>(d * s);
  // g: the element of route k's expert; of routes to the same one the first has it
  const int name = id >= 0 ? id : -1 - sl;
  bool same = twice<16>(name, name);
  if constexpr (SEG == 32) {
    const int other = __shfl_xor(name, 16);
    same |= name == other || twice<32>(name, other);
  }
  if (__ballot(same)) {
    double all = 0.0;
    bool later = false;
    for (int k = 0; k < a.K; ++k) {
      const int other = __shfl(id, k, SEG);
      const double dk = __shfl(d, k, SEG);
      all += other == id ? dk : 0.0;
      later |= other == id && k < sl;
    }
    d = all;
    if (later) id = -1;
  }
  const float g = static_cast<float>(SIG ? d * s * off : s * (d - dot));
  const float rest = static_cast<float>(-dot * inv);          // times its exponential: the other experts' elements
  each<kTok>([&](auto i) {
    if (t0 + i >= a.T) return;
    float o[NPL];
    const float ci = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(rest), i * SEG));
    each<NPL>([&](auto j) { o[j] = SIG ? 0.f : p[i][j] * ci; });
    for (int k = 0; k < a.K; ++k) {
      const int e = __builtin_amdgcn_readlane(id, i * SEG + k);
      const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), i * SEG + k));
      each<NPL>([&](auto j) { o[j] = e == e0 + j ? v : o[j]; });
    }
    float* out = d_logits + static_cast<int64_t>(t0 + i) * a.E;
    if (NPL % 4 == 0 && a.vec) {
      if (e0 < a.E)
        for (int j = 0; j < NPL; j += 4)
          *reinterpret_cast<float4*>(out + e0 + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
    } else {
      each<NPL>([&](auto j) {
        if (e0 + j < a.E) out[e0 + j] = o[j];
      });
    }
  });
}

template <int NPL> void launch_seg(const RouteArgs& a, hipStream_t stream) {
  constexpr int kTok = kWaves * (MOE_WAVE / kSeg);
  const int grid = (a.T + kTok - 1) / kTok;
  const size_t shared = static_cast<size_t>(kWaves) * a.E * sizeof(uint64_t);
  if (a.sigmoid) group_topk_seg_kernel<NPL, true><<<grid, kThreads, shared, stream>>>(a);
  else group_topk_seg_kernel<NPL, false><<<grid, kThreads, shared, stream>>>(a);
}

// Whether the four-tokens-a-wave kernel takes this call.
template <int NPL> bool seg_fits(const RouteArgs& a) {
  const int lg = a.group_size / NPL;
  return a.bias && a.K <= kSegK && a.E % NPL == 0 && aligned16(a.logits) && aligned16(a.bias) &&
         (a.n_group == 1 || (a.group_size % NPL == 0 && (lg & (lg - 1)) == 0));
}

template <int NPL> void launch_fw(RouteArgs a, hipStream_t stream) {
  const int grid = (a.T + kWaves - 1) / kWaves;
  a.vec = a.E % NPL == 0 && aligned16(a.logits) && aligned16(a.bias);
  const size_t shared = static_cast<size_t>(kWaves) * a.E * sizeof(uint64_t);
  if (a.sigmoid) {
    if (a.bias) group_topk_kernel<NPL, true, true><<<grid, kThreads, shared, stream>>>(a);
    else group_topk_kernel<NPL, true, false><<<grid, kThreads, shared, stream>>>(a);
  } else {
    if (a.bias) group_topk_kernel<NPL, false, true><<<grid, kThreads, shared, stream>>>(a);
    else group_topk_kernel<NPL, false, false><<<grid, kThreads, shared, stream>>>(a);
  }
}
template <int NPL> void launch_bw(RouteArgs a, const float* dw, float* dl, hipStream_t stream) {
  a.vec = a.E % NPL == 0 && aligned16(dl);
  const bool wide = a.K > 16;
  const int tok = kWaves * (wide ? 2 : 4), grid = (a.T + tok - 1) / tok;
  if (a.sigmoid) {
    if (wide) group_topk_bw_kernel<NPL, true, 32><<<grid, kThreads, 0, stream>>>(a, dw, dl);
    else group_topk_bw_kernel<NPL, true, 16><<<grid, kThreads, 0, stream>>>(a, dw, dl);
  } else {
    if (wide) group_topk_bw_kernel<NPL, false, 32><<<grid, kThreads, 0, stream>>>(a, dw, dl);
    else group_topk_bw_kernel<NPL, false, 16><<<grid, kThreads, 0, stream>>>(a, dw, dl);
  }
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
  MOE_CHECK(E <= kMaxE && K <= kMaxK && T <= kMaxRows && n_group <= MOE_WAVE && E % n_group == 0, MOE_ERR_UNSUPPORTED);
  MOE_CHECK(K <= topk_group * (E / n_group), MOE_ERR_INVALID_ARG);
  MOE_CHECK(route_scale == route_scale && fabsf(route_scale) < INFINITY, MOE_ERR_INVALID_ARG);
  if (T == 0) return MOE_OK;
  MOE_CHECK(logits && topk_ids && topk_weights, MOE_ERR_INVALID_ARG);
  RouteArgs a{logits, bias, T, E, K, score == MOE_SCORE_SIGMOID, n_group, topk_group, group_top, E / n_group,
              renorm ? 1 : 0, route_scale, 0, topk_ids, topk_weights};
  // Four tokens a wave from 5120 tokens on, where they fill the card: wave per
  // token against four tokens a wave, us, E = 256, K = 8, 4 of 8 groups: 128
  // tokens 4.5 / 5.9, 2048: 8.5 / 9.4, 4096: 9.6 / 9.5, 8192: 13.7 / 12.0, 65536:
  // 58 / 32; E = 128, K = 6: 4096: 6.6 / 6.9, 8192: 8.9 / 7.6, 65536: 41 / 20.
  constexpr int kSegFrom = 5120;
  return in_slices(T, MOE_WAVE, [&](int64_t t, int rows) {
    a.logits = logits + t * E;
    a.T = rows;
    a.ids = topk_ids + t * K;
    a.weights = topk_weights + t * K;
    if (T >= kSegFrom && E > 128 && E <= 256 && seg_fits<16>(a)) launch_seg<16>(a, stream);
    else if (T >= kSegFrom && E > 64 && E <= 128 && seg_fits<8>(a)) launch_seg<8>(a, stream);
    else if (E <= 64) launch_fw<1>(a, stream);
    else if (E <= 128) launch_fw<2>(a, stream);
    else if (E <= 256) launch_fw<4>(a, stream);
    else if (E <= 512) launch_fw<8>(a, stream);
    else launch_fw<16>(a, stream);
  });
}

extern "C" moe_status moe_router_group_topk_backward(const float* logits, const int32_t* topk_ids,
                                                     const float* d_weights, int T, int E, int K, moe_score score,
                                                     int renorm, float route_scale, float* d_logits,
                                                     hipStream_t stream) {
  MOE_CHECK(T >= 0 && E >= 1 && K >= 1 && K <= E, MOE_ERR_INVALID_ARG);
  MOE_CHECK(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID, MOE_ERR_INVALID_ARG);
  MOE_CHECK(E <= kMaxE && K <= kMaxK && T <= kMaxRows, MOE_ERR_UNSUPPORTED);
  MOE_CHECK(route_scale == route_scale && fabsf(route_scale) < INFINITY, MOE_ERR_INVALID_ARG);
  if (T == 0) return MOE_OK;
  MOE_CHECK(logits && topk_ids && d_weights && d_logits && d_logits != logits, MOE_ERR_INVALID_ARG);
  RouteArgs a{};
  a.E = E;
  a.K = K;
  a.sigmoid = score == MOE_SCORE_SIGMOID;
  a.renorm = renorm ? 1 : 0;
  a.scale = route_scale;
  return in_slices(T, MOE_WAVE / 2, [&](int64_t t, int rows) {
    a.logits = logits + t * E;
    a.T = rows;
    a.ids = const_cast<int32_t*>(topk_ids) + t * K;
    const float* dw = d_weights + t * K;
    float* dl = d_logits + t * E;
    if (E <= 64) launch_bw<1>(a, dw, dl, stream);
    else if (E <= 128) launch_bw<2>(a, dw, dl, stream);
    else if (E <= 256) launch_bw<4>(a, dw, dl, stream);
    else if (E <= 512) launch_bw<8>(a, dw, dl, stream);
    else launch_bw<16>(a, dw, dl, stream);
  });
}
