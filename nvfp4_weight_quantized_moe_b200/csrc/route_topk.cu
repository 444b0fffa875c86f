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
// is exact.  With a bias, or with sums of two scores, c is computed in FP32 and
// neighbours in the order that are closer than its error bound send the row
// through the same selection in FP64 (a few rows in a thousand): FP32 alone
// would order about one row in 5000 of a 256-expert router differently.
//
// One warp per token: lane i holds experts i, i + 32, ...; maxima and minima are
// single redux instructions on order-preserving integer keys; lane s holds
// choice s, so topk <= 32 and num_groups <= 32.  The work is one read of the
// logits; per token it is a chain of topk dependent warp reductions, hidden by
// the other warps of the SM for large batches.

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

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  uint64_t ld;
  uint32_t M;
  int E, topk, groups, topk_groups, group_top, group_size;
  int softmax, renorm;
  float scale;
};

// The chosen experts of one row: lane s gets choice s (id, or -1) and its logit.
struct Choice {
  int id;
  float logit;
};

// The selection in the arithmetic of F.  l[j] is the logit of expert 32 j + lane
// (-infinity: not choosable), lmax and zinv the softmax's maximum and 1 / sum.
// `near` reports that two values whose order matters lie within the FP32 error
// bound of each other; F = double never reports it.
template <typename F, int EPL>
NVM_DEV Choice select_experts(const RouteArgs& a, const float (&l)[EPL], F lmax, F zinv, bool& near) {
  using Key = typename KeyOf<F>::type;
  const int lane = threadIdx.x & 31;
  const bool scored = a.bias != nullptr;          // the choice is s + bias; else the logit
  const bool group_scored = scored || a.group_top > 1;
  // FP32 error of s: at most 2^-19 of the largest score (exp and the quotient a
  // few 2^-24 each, a sum of at most 32 terms per lane and 5 tree steps, the
  // rounding of l - lmax weighed by exp(l - lmax)), for softmax 1 / sum at most
  // and 1 for sigmoid; of the sum s + bias: 2^-24 of its value.  The bound
  // compared with covers the errors of both neighbours.
  const float smax = a.softmax ? (float)zinv : 1.0f;
  auto bound = [&](float v) { return smax * 0x1p-18f + fabsf(v) * 0x1p-22f; };
  auto score = [&](float x) -> F {
    if (a.softmax) return exp_f((F)x - lmax) * zinv;
    return (F)1 / ((F)1 + exp_f(-(F)x));
  };

  Key key[EPL];
  float b[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = 32 * j + lane;
    key[j] = 0;
    b[j] = 0.0f;
    if (l[j] == -INFINITY) continue;
    if (scored) {
      b[j] = __ldg(a.bias + e);
      const F c = score(l[j]) + (F)b[j];
      if (c > -(F)INFINITY) key[j] = order_key(c);  // false for NaN too
    } else {
      key[j] = order_key((F)l[j]);
    }
  }

  if (a.groups > 1) {
    // Lane g gets the score of group g: its best value, or the sum of the best
    // two (of the one, where only one can be chosen).
    F mine = -(F)INFINITY;
    bool some = false;
    for (int g = 0; g < a.groups; ++g) {
      const int lo = g * a.group_size, hi = lo + a.group_size;
      Key k1 = 0, k2 = 0;  // this lane's best two
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = 32 * j + lane;
        Key k = 0;
        if (e >= lo && e < hi && key[j] != 0) k = scored || !group_scored ? key[j] : order_key(score(l[j]));
        const Key lower = k < k1 ? k : k1;
        k1 = k > k1 ? k : k1;
        k2 = lower > k2 ? lower : k2;
      }
      const Key best = warp_max_key(k1);
      F v = best != 0 ? key_value(best, F()) : -(F)INFINITY;
      if (a.group_top > 1 && best != 0) {
        const unsigned at = __ballot_sync(kFull, k1 == best);
        const Key next = warp_max_key(lane == __ffs(at) - 1 ? k2 : k1);
        if (next != 0) v += key_value(next, F());
      }
      if (lane == g) {
        mine = v;
        some = best != 0;
      }
    }
    // Rank of this lane's group; a group's rank counts the better ones.
    int rank = 0;
    F above = (F)INFINITY, below = -(F)INFINITY;  // nearest neighbours across the border
    const bool kept_before = some;
    for (int g = 0; g < a.groups; ++g) {
      const F v = __shfl_sync(kFull, mine, g);
      const bool there = __shfl_sync(kFull, (int)some, g) != 0;
      if (there && (v > mine || (v == mine && g < lane))) ++rank;
    }
    const bool kept = kept_before && rank < a.topk_groups;
    const unsigned kept_mask = __ballot_sync(kFull, kept);
    if (sizeof(F) == 4 && group_scored) {
      // The worst kept against the best left out.
      above = kept ? mine : (F)INFINITY;
      below = some && !kept ? mine : -(F)INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const F x = __shfl_xor_sync(kFull, above, o), y = __shfl_xor_sync(kFull, below, o);
        above = x < above ? x : above;
        below = y > below ? y : below;
      }
      if (above - below <= (F)(a.group_top * bound((float)above))) near = true;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (key[j] != 0 && ((kept_mask >> ((32 * j + lane) / a.group_size)) & 1u) == 0) key[j] = 0;
  }

  // topk times: the best key, ties to the lowest expert.  A lane keeps the best
  // of its own experts; the lane whose expert was taken looks again.
  Choice mine{-1, 0.0f};
  Key best = 0;
  int best_e = INT_MAX;
  float best_l = 0.0f, best_b = 0.0f;
  auto look = [&]() {
    best = 0;
    best_e = INT_MAX;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (key[j] > best) {
        best = key[j];
        best_e = 32 * j + lane;
        best_l = l[j];
        best_b = b[j];
      }
  };
  look();
  const bool watch = sizeof(F) == 4 && scored;
  const int picks = watch ? a.topk + 1 : a.topk;  // one more: the best left out
  float last = 0.0f, last_l = 0.0f, last_b = 0.0f;
  for (int s = 0; s < picks; ++s) {
    const Key top = warp_max_key(best);
    if (top == 0) break;
    const int e = __reduce_min_sync(kFull, best == top ? best_e : INT_MAX);
    const float el = __shfl_sync(kFull, best_l, e & 31);
    if (watch) {
      const float eb = __shfl_sync(kFull, best_b, e & 31);
      const float v = (float)key_value(top, F());
      // Equal logits and biases are equal in any arithmetic.
      if (s > 0 && last - v <= bound(last) && !(el == last_l && eb == last_b)) near = true;
      last = v;
      last_l = el;
      last_b = eb;
    }
    if (s < a.topk && lane == s) mine = Choice{e, el};
    if (best_e == e) {
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (32 * j + lane == e) key[j] = 0;
      look();
    }
  }
  return mine;
}

// The FP64 form, out of line: rows whose FP32 order is not certain.
template <int EPL>
__device__ __noinline__ Choice select_exactly(const RouteArgs& a, const float (&l)[EPL], float lmax) {
  double zinv = 0.0;
  if (a.softmax) {
    double z = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) z += exp((double)l[j] - (double)lmax);
    zinv = 1.0 / warp_sum(z);
  }
  bool near = false;
  return select_experts<double, EPL>(a, l, (double)lmax, zinv, near);
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

}  // namespace

template <typename T, int EPL>
__global__ void __launch_bounds__(256) route_topk_kernel(const RouteArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.M) return;
  const T* row = static_cast<const T*>(a.logits) + (uint64_t)t * a.ld;

  // A NaN logit counts as -infinity (not choosable), +infinity as the largest
  // finite value.
  float l[EPL];
  T raw[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    if (32 * j + lane < a.E) raw[j] = __ldg(row + 32 * j + lane);
  float lmax = -INFINITY;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    float v = -INFINITY;
    if (32 * j + lane < a.E) v = logit_f32<T>(raw[j]);
    l[j] = v != v ? -INFINITY : fminf(v, FLT_MAX);
    lmax = fmaxf(lmax, l[j]);
  }
  lmax = warp_max(lmax);

  // Softmax's 1 / sum: needed for the scores as such, not for renormalised
  // weights or a choice by logits.
  const bool scored = a.bias != nullptr || (a.groups > 1 && a.group_top > 1);
  float zinv = 0.0f;
  if (a.softmax && (scored || !a.renorm) && lmax != -INFINITY) {
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) z += expf(l[j] - lmax);
    zinv = 1.0f / warp_sum(z);
  }

  bool near = false;
  Choice c = select_experts<float, EPL>(a, l, lmax, zinv, near);
  if (near) c = select_exactly<EPL>(a, l, lmax);

  // Weights.  Renormalised ones are formed relative to the largest chosen
  // logit, so they are never 0 / 0: softmax exp(l - top); sigmoid
  // exp(l - base) / (1 + exp(l)) with base = min(0, top).
  const bool there = c.id >= 0;
  float w = 0.0f;
  if (a.renorm) {
    const float top = warp_max(there ? c.logit : -INFINITY);
    if (there) {
      if (a.softmax) {
        w = expf(c.logit - top);
      } else if (c.logit > 0.0f) {
        w = 1.0f / (1.0f + expf(-c.logit));
      } else {
        w = expf(c.logit - fminf(0.0f, top)) / (1.0f + expf(c.logit));
      }
    }
    const float sum = warp_sum(w);
    if (there) w = w / sum;
  } else if (there) {
    if (a.softmax) {
      w = expf(c.logit - lmax) * zinv;
    } else if (c.logit > 0.0f) {
      w = 1.0f / (1.0f + expf(-c.logit));
    } else {
      const float x = expf(c.logit);
      w = x / (1.0f + x);
    }
  }
  if (lane < a.topk) {
    const uint64_t at = (uint64_t)t * a.topk + lane;
    a.ids[at] = c.id;
    a.weights[at] = w * a.scale;
  }
}

namespace {

template <typename T>
cudaError_t launch_route_topk_of(const RouteArgs& a, cudaStream_t stream) {
  // One warp per CTA while that leaves every SM at most a few tokens (their
  // chains then run on separate schedulers), eight for large batches.
  const int warps = a.M <= 592 ? 1 : 8;
  const dim3 grid((a.M + warps - 1) / warps), block(32 * warps);
  const int epl = (a.E + 31) / 32;
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
  a.group_size = (int)(r.num_experts / r.num_groups);
  a.softmax = r.softmax;
  a.renorm = r.renormalize;
  a.scale = r.scale;
  return logits_f32 ? launch_route_topk_of<float>(a, stream) : launch_route_topk_of<uint16_t>(a, stream);
}

}  // namespace nvm
