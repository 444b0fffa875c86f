// Routing of tokens to experts: scores of the router's logits, a balance bias,
// groups of experts, the topk best and their weights, in the layout that the
// route sort and the forward take (topk_ids, topk_weights).
//
//   s[e] = softmax_e(l) or 1 / (1 + exp(-l[e]));   c[e] = s[e] + bias[e]
//   group score = its best c, or the sum of its two best; the topk_groups best
//   groups stay; the topk best c of what stays, descending; weights from s.
//
// Every comparison goes by the exact values, ties to the lower index.  Without
// a bias the choice is made on the logits themselves (s is monotone in l), which
// is exact.  With a bias, or with sums of two scores, c is computed in FP32, and
// a row in which two values whose order matters are closer than the error bound
// goes through the same selection once more in FP64: about one row in 1000 of a
// 256-expert router, where FP32 alone would order one in 5000 differently.
//
// One warp per token.  Lane i holds ceil(E / 32) consecutive experts, so a
// lower lane means a lower index, a tie is settled by the lowest set bit of a
// ballot, and where a group is whole lanes the best two of all groups are found
// at once by a butterfly inside the group's lanes.  Maxima are single redux
// instructions on order-preserving integer keys.  Lane s ends up with choice s,
// so topk <= 32 and num_groups <= 32.  The work is one read of the logits; per
// token it is a chain of topk dependent warp reductions, hidden by the other
// warps of the SM for large batches.

#include <cfloat>
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace nvm {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// Order-preserving integer keys; 0 marks an expert that cannot be chosen (every
// finite value and +infinity has a larger key).
NVM_DEV uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 and +0 are the same value
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
NVM_DEV uint64_t order_key(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
NVM_DEV float key_value(uint32_t k, float) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
NVM_DEV double key_value(uint64_t k, double) {
  return __longlong_as_double((long long)(k & 0x8000000000000000ull ? k ^ 0x8000000000000000ull : ~k));
}
template <typename F>
struct KeyOf;
template <>
struct KeyOf<float> {
  using type = uint32_t;
};
template <>
struct KeyOf<double> {
  using type = uint64_t;
};

NVM_DEV uint32_t warp_max_key(uint32_t k) { return __reduce_max_sync(kFull, k); }
NVM_DEV uint64_t warp_max_key(uint64_t k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t t = __shfl_xor_sync(kFull, k, o);
    k = t > k ? t : k;
  }
  return k;
}

NVM_DEV float exp_f(float v) { return expf(v); }
NVM_DEV double exp_f(double v) { return exp(v); }

template <typename F>
NVM_DEV F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

constexpr int kMaxWarps = 8;

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  uint64_t ld;
  uint32_t M;
  int E, per_lane;  // per_lane = ceil(E / 32)
  int topk, groups, topk_groups, group_top;
  int group_lanes;       // lanes of a group, if groups are whole lanes; else 0
  uint32_t group_magic;  // ceil(2^20 / group size): expert e is in group e * magic >> 20
  int softmax, renorm;
  int vec;               // rows can be read 16 bytes (bf16 of 128 experts: 8) at a time
  float scale;
};

// exp for scores that are only compared (FP32: the hardware exponential) ...
NVM_DEV float exp_near(float v) { return __expf(v); }
NVM_DEV double exp_near(double v) { return exp(v); }
NVM_DEV float recip_near(float v) { return __fdividef(1.0f, v); }
NVM_DEV double recip_near(double v) { return 1.0 / v; }

// The selection in the arithmetic of F: the chosen experts, best first, into
// picks[0 .. topk) (-1 where none is left).  l[j] is the logit of expert
// per_lane * lane + j (-infinity: not choosable), lmax and zinv the softmax's
// maximum and 1 / sum.  Returns whether two values whose order matters lie within
// the FP32 error bound of each other (never for F = double).
template <typename F, int EPL>
NVM_DEV bool select_experts(const RouteArgs& a, const float (&l)[EPL], F lmax, F zinv, int* picks) {
  using Key = typename KeyOf<F>::type;
  constexpr bool kFast = sizeof(F) == 4;
  constexpr int kUnroll = kFast ? EPL : 1;  // FP64 is rare: small code, few registers
  const int lane = threadIdx.x & 31, e0 = lane * a.per_lane;
  const bool scored = a.bias != nullptr;  // the choice is s + bias; else the logit
  // Error of an FP32 s.  Sigmoid: the exponential is off by (2 + 1.2 |x|) 2^-23 of
  // its value, which s (1 - s) weighs to under 2^-23; 1 + exp and the quotient add
  // 2^-24 and 2^-22: under 2^-21.  Softmax, in units of the largest score 1 / sum:
  // the difference and the exponential as much, the sum EPL + 5 roundings.  s + bias
  // adds 2^-24 of its value.  Twice that for two neighbours.
  const float unit = a.softmax ? (float)zinv * (8 + 2 * (EPL + 5)) * 0x1p-23f : 0x1p-20f;
  auto bound = [&](float v) { return unit + fabsf(v) * 0x1p-23f; };
  auto score = [&](float x) -> F {
    if (a.softmax) return exp_near((F)x - lmax) * zinv;
    return recip_near((F)1 + exp_near(-(F)x));
  };

  Key key[EPL];
#pragma unroll kUnroll
  for (int j = 0; j < EPL; ++j) {
    key[j] = 0;
    if (l[j] == -INFINITY) continue;
    F c = (F)l[j];
    if (scored) c = score(l[j]) + (F)__ldg(a.bias + e0 + j);
    if (c > -(F)INFINITY) key[j] = order_key(c);  // false for NaN too
  }

  bool near = false;
  if (a.groups > 1) {
    // Lane g gets the score of group g: its best value, or the sum of its best two
    // (of the one, where only one can be chosen); key 0: no expert to choose.
    const bool sums = a.group_top > 1;
    auto value_key = [&](int j) -> Key {
      return key[j] == 0 || scored || !sums ? key[j] : order_key(score(l[j]));
    };
    auto total = [&](Key k1, Key k2) -> Key {
      if (k1 == 0 || k2 == 0 || !sums) return k1;
      return order_key(key_value(k1, F()) + key_value(k2, F()));
    };
    Key mine = 0;
    if (a.group_lanes > 0) {
      Key k1 = 0, k2 = 0;
#pragma unroll kUnroll
      for (int j = 0; j < EPL; ++j) {
        const Key k = value_key(j), lower = k < k1 ? k : k1;
        k1 = k > k1 ? k : k1;
        k2 = lower > k2 ? lower : k2;
      }
      for (int o = 1; o < a.group_lanes; o <<= 1) {
        const Key p1 = __shfl_xor_sync(kFull, k1, o), p2 = __shfl_xor_sync(kFull, k2, o);
        const Key lower = p1 < k1 ? p1 : k1, second = p2 > k2 ? p2 : k2;
        k1 = p1 > k1 ? p1 : k1;
        k2 = lower > second ? lower : second;
      }
      mine = __shfl_sync(kFull, total(k1, k2), lane * a.group_lanes & 31);
      if (lane >= a.groups) mine = 0;
    } else {
#pragma unroll 1
      for (int g = 0; g < a.groups; ++g) {
        Key k1 = 0, k2 = 0;  // this lane's best two
#pragma unroll kUnroll
        for (int j = 0; j < EPL; ++j) {
          if (key[j] == 0 || (int)((uint32_t)(e0 + j) * a.group_magic >> 20) != g) continue;
          const Key k = value_key(j), lower = k < k1 ? k : k1;
          k1 = k > k1 ? k : k1;
          k2 = lower > k2 ? lower : k2;
        }
        const Key best = warp_max_key(k1);
        const unsigned at = __ballot_sync(kFull, k1 == best);
        const Key next = warp_max_key(lane == __ffs(at) - 1 ? k2 : k1);
        if (lane == g) mine = total(best, next);
      }
    }
    // A group's rank counts the better ones.
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
      const Key v = __shfl_sync(kFull, mine, g);
      rank += v > mine || (v == mine && g < lane);
    }
    const bool kept = mine != 0 && rank < a.topk_groups;
    const unsigned kept_mask = __ballot_sync(kFull, kept);
    if constexpr (kFast) {
      // The worst kept against the best left out (there may be none).
      const Key above = __reduce_min_sync(kFull, kept ? mine : 0xffffffffu);
      const Key below = __reduce_max_sync(kFull, kept ? 0u : mine);
      if ((scored || sums) && below != 0) {
        const float v = key_value(above, F());
        near = v - key_value(below, F()) <= a.group_top * bound(v);
      }
    }
    if (a.group_lanes > 0) {
      if (((kept_mask >> (lane / a.group_lanes)) & 1u) == 0) {
#pragma unroll kUnroll
        for (int j = 0; j < EPL; ++j) key[j] = 0;
      }
    } else {
#pragma unroll kUnroll
      for (int j = 0; j < EPL; ++j)
        if (key[j] != 0 && ((kept_mask >> ((uint32_t)(e0 + j) * a.group_magic >> 20)) & 1u) == 0) key[j] = 0;
    }
  }

  // topk times the best key of the warp.  A lane keeps the best of its own experts;
  // the lane whose expert was taken looks again.  One more round, where
  // neighbours are watched, for the best left out.
  if (lane < a.topk) picks[lane] = -1;
  __syncwarp();
  const bool watch = kFast && scored;
  const int rounds = watch ? a.topk + 1 : a.topk;
  Key best = 0;
  int best_j = 0;
#pragma unroll kUnroll
  for (int j = 0; j < EPL; ++j)
    if (key[j] > best) {
      best = key[j];
      best_j = j;
    }
  float last = INFINITY;
#pragma unroll 1
  for (int s = 0; s < rounds; ++s) {
    const Key top = warp_max_key(best);
    if (top == 0) break;
    if (watch) {
      const float v = (float)key_value(top, F());
      near |= last - v <= bound(v);  // infinity - infinity is no near pair
      last = v;
    }
    const unsigned at = __ballot_sync(kFull, best == top);
    if (lane == __ffs(at) - 1) {
      if (s < a.topk) picks[s] = e0 + best_j;
      best = 0;
      const int taken = best_j;
#pragma unroll kUnroll
      for (int j = 0; j < EPL; ++j) {
        if (j == taken) key[j] = 0;
        if (key[j] > best) {
          best = key[j];
          best_j = j;
        }
      }
    }
  }
  __syncwarp();
  return near;
}

template <typename T>
NVM_DEV float logit_f32(T v);
template <>
NVM_DEV float logit_f32(float v) {
  return v;
}
template <>
NVM_DEV float logit_f32(uint16_t v) {
  return bf16_bits_to_f32(v);
}

// A NaN logit counts as -infinity (not choosable), +infinity as the largest
// finite value.
NVM_DEV float clean_logit(float v) { return v != v ? -INFINITY : fminf(v, FLT_MAX); }

template <typename T, int EPL>
NVM_DEV void load_logits(const RouteArgs& a, const T* row, float (&l)[EPL]) {
  constexpr int kPer = 16 / sizeof(T) < EPL ? 16 / sizeof(T) : EPL;  // elements of one load
  const int e0 = (threadIdx.x & 31) * a.per_lane;
  if (a.vec) {  // per_lane == EPL, E == 32 EPL
    struct alignas(kPer * sizeof(T)) Piece {
      T v[kPer];
    };
    Piece p[EPL / kPer];
#pragma unroll
    for (int i = 0; i < EPL / kPer; ++i) p[i] = reinterpret_cast<const Piece*>(row + e0)[i];
#pragma unroll
    for (int j = 0; j < EPL; ++j) l[j] = clean_logit(logit_f32<T>(p[j / kPer].v[j % kPer]));
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      l[j] = -INFINITY;
      if (j < a.per_lane && e0 + j < a.E) l[j] = clean_logit(logit_f32<T>(__ldg(row + e0 + j)));
    }
  }
}

// The FP64 selection of a row whose FP32 order is not certain, out of line; it
// reads the row again, so nothing has to be kept for it.
template <typename T, int EPL>
__device__ __noinline__ void select_exactly(const RouteArgs& a, const T* row, float lmax, int* picks) {
  float l[EPL];
  load_logits<T, EPL>(a, row, l);
  double zinv = 0.0;
  if (a.softmax) {
    double z = 0.0;
    for (int j = 0; j < EPL; ++j) z += exp((double)l[j] - (double)lmax);
    zinv = 1.0 / warp_sum(z);
  }
  select_experts<double, EPL>(a, l, (double)lmax, zinv, picks);
}

}  // namespace

template <typename T, int EPL>
__global__ void __launch_bounds__(32 * kMaxWarps, EPL <= 8 ? 4 : EPL == 16 ? 2 : 1) route_topk_kernel(const RouteArgs a) {
  __shared__ int s_picks[kMaxWarps][32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.M) return;
  const T* row = static_cast<const T*>(a.logits) + (uint64_t)t * a.ld;
  int* picks = s_picks[threadIdx.x >> 5];

  float l[EPL];
  load_logits<T, EPL>(a, row, l);
  // Softmax's maximum, and 1 / sum where the scores as such are needed: not for
  // renormalised weights or a choice by logits.
  float lmax = 0.0f, zinv = 0.0f;
  if (a.softmax) {
    lmax = l[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) lmax = fmaxf(lmax, l[j]);
    lmax = key_value(__reduce_max_sync(kFull, order_key(lmax)), 0.0f);
    if (lmax != -INFINITY && (a.bias != nullptr || a.group_top > 1 || !a.renorm)) {
      float z = 0.0f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) z += expf(l[j] - lmax);
      zinv = 1.0f / warp_sum(z);
    }
  }
  if (select_experts<float, EPL>(a, l, lmax, zinv, picks)) select_exactly<T, EPL>(a, row, lmax, picks);

  // Weights.  Renormalised ones are formed relative to the largest chosen
  // logit, so they are never 0 / 0: softmax exp(l - top); sigmoid
  // exp(l - base) / (1 + exp(l)) with base = min(0, top).
  const int id = lane < a.topk ? picks[lane] : -1;
  const float x = id >= 0 ? clean_logit(logit_f32<T>(__ldg(row + id))) : -INFINITY;
  float base = a.softmax ? lmax : 0.0f;
  if (a.renorm) {
    base = key_value(__reduce_max_sync(kFull, order_key(x)), 0.0f);
    if (!a.softmax) base = fminf(base, 0.0f);
  }
  float w = 0.0f;
  if (id >= 0) {
    const float low = expf(fminf(x, a.softmax ? x : 0.0f) - base);
    w = low;
    if (!a.softmax) w = x > 0.0f ? 1.0f / (1.0f + expf(-x)) : low / (1.0f + expf(x));
  }
  float norm = a.softmax ? zinv : 1.0f;
  if (a.renorm) norm = 1.0f / warp_sum(w);
  if (lane < a.topk) {
    const uint64_t at = (uint64_t)t * a.topk + lane;
    a.ids[at] = id;
    a.weights[at] = id >= 0 ? w * norm * a.scale : 0.0f;
  }
}

namespace {

template <typename T>
cudaError_t launch_route_topk_of(const RouteArgs& a, cudaStream_t stream) {
  // One warp per CTA while that leaves every SM at most a few tokens (their
  // chains then run on separate schedulers), eight for large batches.
  const int warps = a.M <= 592 ? 1 : kMaxWarps;
  const dim3 grid((a.M + warps - 1) / warps), block(32 * warps);
  const int epl = a.per_lane;
  if (epl <= 1) return launch_pdl(route_topk_kernel<T, 1>, grid, block, 0, stream, a);
  if (epl <= 2) return launch_pdl(route_topk_kernel<T, 2>, grid, block, 0, stream, a);
  if (epl <= 4) return launch_pdl(route_topk_kernel<T, 4>, grid, block, 0, stream, a);
  if (epl <= 8) return launch_pdl(route_topk_kernel<T, 8>, grid, block, 0, stream, a);
  if (epl <= 16) return launch_pdl(route_topk_kernel<T, 16>, grid, block, 0, stream, a);
  return launch_pdl(route_topk_kernel<T, 32>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_route_topk(const void* logits, bool logits_f32, uint64_t ld, uint32_t num_tokens,
                              const RouterConfig& r, int32_t* ids, float* weights, cudaStream_t stream) {
  RouteArgs a{};
  a.logits = logits;
  a.bias = r.bias;
  a.ids = ids;
  a.weights = weights;
  a.ld = ld;
  a.M = num_tokens;
  a.E = (int)r.num_experts;
  a.topk = (int)r.topk;
  a.groups = (int)r.num_groups;
  a.topk_groups = (int)r.topk_groups;
  a.group_top = (int)r.group_top;
  const uint32_t group_size = r.num_experts / r.num_groups;
  a.per_lane = (a.E + 31) / 32;
  a.group_magic = ((1u << 20) + group_size - 1) / group_size;
  if (r.num_experts % 32 == 0 && 32 % r.num_groups == 0) a.group_lanes = 32 / a.groups;
  // Wide reads: whole lanes of a power of two of experts, on 16 bytes (or on the
  // lane's bytes, where they are fewer).
  const uint32_t lane_bytes = (uint32_t)a.per_lane * (logits_f32 ? 4 : 2), piece = lane_bytes < 16 ? lane_bytes : 16;
  a.vec = r.num_experts % 32 == 0 && (a.per_lane & (a.per_lane - 1)) == 0 &&
          reinterpret_cast<uintptr_t>(logits) % piece == 0 && ld * (logits_f32 ? 4 : 2) % piece == 0;
  a.softmax = r.softmax;
  a.renorm = r.renormalize;
  a.scale = r.scale;
  return logits_f32 ? launch_route_topk_of<float>(a, stream) : launch_route_topk_of<uint16_t>(a, stream);
}

}  // namespace nvm
