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
// where two values whose order matters are closer than its error bound, they are
// computed again in FP64: in about one row in 1000 of a 256-expert router, where
// FP32 alone would order one in 5000 differently.
//
// One warp per token.  Lane i holds ceil(E / 32) consecutive experts, so a
// lower lane means a lower index, a tie is settled by the lowest set bit of a
// ballot, and where a group is whole lanes the best two of all groups are found
// at once by a butterfly inside the group's lanes.  Maxima are single redux
// instructions on order-preserving integer keys.  Lane s ends up with choice s,
// so topk <= 32 and num_groups <= 32.
//
// The work is one read of the logits (8191 x 256 FP32: 1.4 us at the copy
// bandwidth); what bounds it is instruction issue, about 910 warp instructions a
// token with scores, bias and groups (8191 x 256: 13 us, 70 % of the issue slots),
// 600 without (8192 x 128 BF16: 7.7 us), and for one token the chain of warp
// reductions (2.0 us and 3.5 us with groups, of which 1.3 us are the launch).

#include <cfloat>
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace nvm {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// Order-preserving integer keys.  An expert can be chosen if its key is above
// that of -infinity; 0 marks one that was taken or whose group was left out.
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
  static constexpr uint32_t none = 0x007fffffu;  // of -infinity
};
template <>
struct KeyOf<double> {
  using type = uint64_t;
  static constexpr uint64_t none = 0x000fffffffffffffull;
};
NVM_DEV float or_minus_infinity(float v) { return fmaxf(v, -INFINITY); }  // NaN to -infinity
NVM_DEV double or_minus_infinity(double v) { return fmax(v, -(double)INFINITY); }

NVM_DEV uint32_t warp_max_key(uint32_t k) { return __reduce_max_sync(kFull, k); }
NVM_DEV uint64_t warp_max_key(uint64_t k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t t = __shfl_xor_sync(kFull, k, o);
    k = t > k ? t : k;
  }
  return k;
}

template <typename F>
NVM_DEV F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

constexpr int kMaxWarps = 4;

// 2^x and 1 / x as the hardware has them (2^-22 off, results below the normal
// range 0), for scores that are only compared.
NVM_DEV float exp2_near(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
NVM_DEV float recip_near(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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
  int vec_bias;          // so can the bias
  float scale;
};

// What a warp's selection leaves in shared memory.
struct alignas(16) Picks {
  int id[32];           // the chosen experts, best first; -1 where none is left
  float logit[32];      // their logits, where the choice is by logits
  uint32_t key[32];     // candidates in the order of their index: keys (0 past them)
  int expert[32];       // ... and experts
  uint2 ranked[32];     // the best of them, best first (key, expert)
};

// The groups of a row and the lanes' experts: expert e's group, or whether it stays.
NVM_DEV bool in_mask(const RouteArgs& a, uint32_t mask, int e) {
  return ((mask >> ((uint32_t)e * a.group_magic >> 20)) & 1u) != 0;
}

// A group's two best choice keys.
template <typename Key>
struct Best2 {
  Key one, two;
};

// Lane g gets those of group g from `value`, the choice keys of the lane's experts;
// the second one only where a group's score needs it.
template <typename F, int EPL, typename Value>
NVM_DEV Best2<typename KeyOf<F>::type> best_two(const RouteArgs& a, Value value) {
  using Key = typename KeyOf<F>::type;
  constexpr int kUnroll = sizeof(F) == 4 ? EPL : 1;
  const int lane = threadIdx.x & 31, e0 = lane * a.per_lane;
  Best2<Key> mine{0, 0};
  if (a.group_lanes > 0) {
    Key k1 = 0, k2 = 0;
#pragma unroll kUnroll
    for (int j = 0; j < EPL; ++j) {
      const Key k = value(j), lower = k < k1 ? k : k1;
      k1 = k > k1 ? k : k1;
      k2 = lower > k2 ? lower : k2;
    }
#pragma unroll 1
    for (int o = 1; o < a.group_lanes; o <<= 1) {
      const Key p1 = __shfl_xor_sync(kFull, k1, o), p2 = __shfl_xor_sync(kFull, k2, o);
      const Key lower = p1 < k1 ? p1 : k1, second = p2 > k2 ? p2 : k2;
      k1 = p1 > k1 ? p1 : k1;
      k2 = lower > second ? lower : second;
    }
    const int from = lane * a.group_lanes & 31;
    k1 = __shfl_sync(kFull, k1, from);
    if (a.group_top > 1) k2 = __shfl_sync(kFull, k2, from);
    if (lane < a.groups) mine = {k1, k2};
    return mine;
  }
#pragma unroll 1
  for (int g = 0; g < a.groups; ++g) {
    Key k1 = 0, k2 = 0;  // this lane's best two
#pragma unroll kUnroll
    for (int j = 0; j < EPL; ++j) {
      if ((int)((uint32_t)(e0 + j) * a.group_magic >> 20) != g) continue;
      const Key k = value(j), lower = k < k1 ? k : k1;
      k1 = k > k1 ? k : k1;
      k2 = lower > k2 ? lower : k2;
    }
    const Key best = warp_max_key(k1);
    const unsigned at = __ballot_sync(kFull, k1 == best);
    const Key next = warp_max_key(lane == __ffs(at) - 1 ? k2 : k1);
    if (lane == g) mine = {best, next};
  }
  return mine;
}

// Whether a group's score is the sum of two values: it is that of the one where only
// one can be chosen.
template <typename F>
NVM_DEV bool is_sum(const RouteArgs& a, Best2<typename KeyOf<F>::type> b) {
  return a.group_top > 1 && b.two > KeyOf<F>::none;
}

// Key of a group's score.  Two values near the type's lowest add up to -infinity in
// FP32; such a group can be chosen, so it counts as the lowest finite one (and is
// ordered in FP64).
NVM_DEV float finite_sum(float x, float y) { return fmaxf(x + y, -FLT_MAX); }
NVM_DEV double finite_sum(double x, double y) { return x + y; }
template <typename F>
NVM_DEV typename KeyOf<F>::type group_key(const RouteArgs& a, Best2<typename KeyOf<F>::type> b) {
  return is_sum<F>(a, b) ? order_key(finite_sum(key_value(b.one, F()), key_value(b.two, F()))) : b.one;
}

// The topk_groups best of the groups' keys, as a mask; a group's rank counts the
// better ones.
template <typename Key>
NVM_DEV unsigned best_groups(const RouteArgs& a, Key mine, Key none) {
  const int lane = threadIdx.x & 31;
  int rank = 0;
#pragma unroll 1
  for (int g = 0; g < a.groups; ++g) {
    const Key v = __shfl_sync(kFull, mine, g);
    rank += v > mine || (v == mine && g < lane);
  }
  return __ballot_sync(kFull, mine > none && rank < a.topk_groups);
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
NVM_DEV float clean_logit(float v) { return fminf(or_minus_infinity(v), FLT_MAX); }

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

// The FP64 forms, for rows that FP32 cannot order: out of line, small, and reading
// the row again, so that the common way keeps nothing for them.
struct Scores64 {
  double lmax, zinv;
};

template <typename T>
__device__ __noinline__ Scores64 scores_exactly(const RouteArgs& a, const T* row, float lmax) {
  Scores64 s{(double)lmax, 0.0};
  if (a.softmax) {
    double z = 0.0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < a.E; e += 32) z += exp((double)clean_logit(logit_f32<T>(row[e])) - s.lmax);
    s.zinv = 1.0 / warp_sum(z);
  }
  return s;
}

// Key of the choice value of expert e.
template <typename T>
__device__ __noinline__ uint64_t choice_exactly(const RouteArgs& a, const T* row, Scores64 s, int e) {
  const float x = clean_logit(logit_f32<T>(row[e]));
  if (x == -INFINITY) return 0;
  const double p = a.softmax ? exp((double)x - s.lmax) * s.zinv : 1.0 / (1.0 + exp(-(double)x));
  return order_key(or_minus_infinity(a.bias != nullptr ? p + (double)a.bias[e] : p));
}

template <typename T, int EPL>
__device__ __noinline__ unsigned groups_exactly(const RouteArgs& a, const T* row, Scores64 s) {
  const int e0 = (threadIdx.x & 31) * a.per_lane;
  const Best2<uint64_t> two = best_two<double, EPL>(a, [&](int j) -> uint64_t {
    return j < a.per_lane && e0 + j < a.E ? choice_exactly<T>(a, row, s, e0 + j) : 0;
  });
  return best_groups(a, group_key<double>(a, two), KeyOf<double>::none);
}

// The whole choice among the experts of the groups of `mask`: topk times the best.
template <typename T, int EPL>
__device__ __noinline__ void pick_exactly(const RouteArgs& a, const T* row, Scores64 s, unsigned mask, Picks& picks) {
  const int lane = threadIdx.x & 31, e0 = lane * a.per_lane;
  uint64_t key[EPL];
#pragma unroll 1
  for (int j = 0; j < EPL; ++j) {
    key[j] = 0;
    if (j < a.per_lane && e0 + j < a.E && in_mask(a, mask, e0 + j)) key[j] = choice_exactly<T>(a, row, s, e0 + j);
  }
#pragma unroll 1
  for (int r = 0; r < a.topk; ++r) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll 1
    for (int j = 0; j < EPL; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    const uint64_t top = warp_max_key(best);
    if (top <= KeyOf<double>::none) break;
    if (lane == __ffs(__ballot_sync(kFull, best == top)) - 1) {
      picks.id[r] = e0 + at;
      key[at] = 0;
    }
  }
  __syncwarp();
}

// The order of the n candidates by their FP64 values.
template <typename T>
__device__ __noinline__ void rank_exactly(const RouteArgs& a, const T* row, Scores64 s, int n, Picks& picks) {
  const int lane = threadIdx.x & 31;
  const int e = lane < n ? picks.expert[lane] : 0;
  const uint64_t key = lane < n ? choice_exactly<T>(a, row, s, e) : 0;
  int rank = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const uint64_t k = __shfl_sync(kFull, key, i);
    rank += k > key || (k == key && i < lane);
  }
  if (lane < n && rank < a.topk) picks.id[rank] = e;
  __syncwarp();
}

// The selection, into picks.id[0 .. topk).  l[j] is the logit of expert per_lane *
// lane + j (-infinity: not choosable), lmax and zinv the softmax's maximum and
// 1 / sum.
template <typename T, int EPL>
NVM_DEV void select_experts(const RouteArgs& a, const T* row, const float (&l)[EPL], float lmax, float zinv,
                            Picks& picks) {
  constexpr uint32_t kNone = KeyOf<float>::none;
  const int lane = threadIdx.x & 31, e0 = lane * a.per_lane;
  const bool scored = a.bias != nullptr;  // the choice is s + bias; else the logit
  // Error of an FP32 s.  Sigmoid: the exponential is off by (2 + 1.2 |x|) 2^-23 of
  // its value (its own error, and the rounded product in its exponent), which
  // s (1 - s) weighs to under 2^-23; 1 + exp and the quotient add 2^-24 and 2^-23:
  // under 2^-21.  Softmax, in units of the largest score 1 / sum:
  // the difference and the exponential as much, the sum EPL + 5 roundings.  s + bias
  // adds 2^-24 of its value.  Twice that for two neighbours.
  const float unit = a.softmax ? zinv * (8 + 2 * (EPL + 5)) * 0x1p-23f : 0x1p-20f;
  auto bound = [&](float v) { return unit + fabsf(v) * 0x1p-23f; };
  auto softmax_score = [&](float x) { return exp2_near((x - lmax) * 1.44269504f) * zinv; };
  auto sigmoid_score = [&](float x) { return recip_near(1.0f + exp2_near(x * -1.44269504f)); };

  uint32_t key[EPL];
  if (scored) {
    float b[EPL];
    if (a.vec_bias) {
      constexpr int kPer = EPL < 4 ? EPL : 4;
      struct alignas(4 * kPer) Piece {
        float v[kPer];
      };
#pragma unroll
      for (int i = 0; i < EPL / kPer; ++i) {
        const Piece p = reinterpret_cast<const Piece*>(a.bias + e0)[i];
#pragma unroll
        for (int j = 0; j < kPer; ++j) b[i * kPer + j] = p.v[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) b[j] = j < a.per_lane && e0 + j < a.E ? __ldg(a.bias + e0 + j) : 0.0f;
    }
    auto choose = [&](auto score) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] = l[j] == -INFINITY ? 0 : order_key(or_minus_infinity(score(l[j]) + b[j]));
    };
    if (a.softmax) choose(softmax_score);
    else choose(sigmoid_score);
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = order_key(l[j]);
  }

  unsigned mask = 1u;
  if (a.groups > 1) {
    const bool sums = a.group_top > 1;
    Best2<uint32_t> two;
    if (scored || !sums) {
      two = best_two<float, EPL>(a, [&](int j) -> uint32_t { return key[j]; });
    } else {
      two = best_two<float, EPL>(a, [&](int j) -> uint32_t {
        if (key[j] <= kNone) return 0;
        return order_key(a.softmax ? softmax_score(l[j]) : sigmoid_score(l[j]));
      });
    }
    // A score is off by its values' errors and, for a sum, its own rounding: all of them
    // by the values' sizes, which a sum of opposite signs does not show.
    const bool sum = is_sum<float>(a, two);
    const float one = key_value(two.one, 0.0f), other = sum ? key_value(two.two, 0.0f) : 0.0f;
    const float v = sum ? finite_sum(one, other) : one;
    uint32_t rest = sum ? order_key(v) : two.one;
    const float of_size = sums ? 0x1.00001p-23f : 0x1.00001p-24f, of_score = sums ? unit : 0.5f * unit;
    const float off = two.one > kNone ? fmaf(fabsf(one) + fabsf(other), of_size, of_score) : 0.0f;
    // The best groups one after another.
    uint32_t worst = 0;
    mask = 0;
#pragma unroll 1
    for (int r = 0; r < a.topk_groups; ++r) {
      const uint32_t top = __reduce_max_sync(kFull, rest);
      if (top <= kNone) break;
      const int at = __ffs(__ballot_sync(kFull, rest == top)) - 1;
      mask |= 1u << at;
      if (lane == at) rest = 0;
      worst = top;
    }
    if (scored || sums) {
      const uint32_t below = __reduce_max_sync(kFull, rest);  // there may be none
      const float from = key_value(worst, 0.0f), gap = from - key_value(below, 0.0f);
      const float most_off = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(off)));
      if (below > kNone && !(gap > 2.00001f * most_off)) {
        // Is the least that any kept group's score can be under the most that a left one's
        // can?  Both as distances from the worst kept one's, exact where they are small;
        // what is not finite may be anywhere.
        const bool bounded = off < INFINITY;
        const uint32_t least = (mask >> lane) & 1u ? order_key(bounded ? v - from - off : -INFINITY) : 0xffffffffu;
        const uint32_t most = rest > kNone ? order_key(bounded ? v - from + off : INFINITY) : 0u;
        if (__reduce_min_sync(kFull, least) <= __reduce_max_sync(kFull, most))
          mask = groups_exactly<T, EPL>(a, row, scores_exactly<T>(a, row, lmax));
      }
    }
    if (a.group_lanes > 0) {
      const uint32_t stays = (mask >> (lane / a.group_lanes)) & 1u ? 0xffffffffu : 0u;
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] &= stays;
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (!in_mask(a, mask, e0 + j)) key[j] = 0;
    }
  }

  // Every one of the topk best experts is at least the topk-th best of the lanes'
  // bests.  Usually few others are (9 of 256 experts for 8): these candidates go
  // to one lane each, and a candidate's rank counts the better ones.  Where FP32
  // is not exact, what is within its error below them is a candidate too.
  picks.id[lane] = -1;
  picks.key[lane] = 0;
  uint32_t best = key[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) best = key[j] > best ? key[j] : best;
  uint32_t floor = 0, rest = best;
#pragma unroll 4
  for (int s = 0; s < a.topk; ++s) {
    floor = __reduce_max_sync(kFull, rest);
    if (rest == floor) rest = 0;
  }
  auto lower = [&](uint32_t from) {
    if (scored) {
      const float v = key_value(from, 0.0f), under = v - bound(v);
      if (under < v) from = order_key(under);  // not of an infinity
    }
    return from > kNone ? from : kNone + 1;
  };
  auto candidates = [&](uint32_t from) {  // of this lane
    int c = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) c += key[j] >= from;
    return c;
  };
  uint32_t bar = lower(floor);
  int count = candidates(bar);
  if (__reduce_add_sync(kFull, count) > 32) {
    // Bisect for a higher bar that topk to 32 experts pass (there is none where
    // too many are equal).
    uint32_t over = __reduce_max_sync(kFull, best) + 1;
    int n = 33;
#pragma unroll 1
    while (over - floor > 1 && n > 32) {
      const uint32_t middle = floor + (over - floor) / 2;
      if ((int)__reduce_add_sync(kFull, candidates(middle)) < a.topk) {
        over = middle;
      } else {
        floor = middle;
        bar = lower(floor);
        count = candidates(bar);
        n = __reduce_add_sync(kFull, count);
      }
    }
  }
  int upto = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += v;
  }
  const int n = __shfl_sync(kFull, upto, 31);
  __syncwarp();
  if (n <= 32) {
    if (count > 0) {
      int at = upto - count;
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (key[j] >= bar) {
          picks.key[at] = key[j];
          picks.expert[at++] = e0 + j;
        }
    }
    __syncwarp();
    const uint2 c = make_uint2(picks.key[lane], (uint32_t)picks.expert[lane]);
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i < n; i += 4) {
      const uint4 k = *reinterpret_cast<const uint4*>(picks.key + i);
      // Equal keys: found in the order of their index.
      rank += k.x > c.x || (k.x == c.x && i < lane);
      rank += k.y > c.x || (k.y == c.x && i + 1 < lane);
      rank += k.z > c.x || (k.z == c.x && i + 2 < lane);
      rank += k.w > c.x || (k.w == c.x && i + 3 < lane);
    }
    if (lane < n && rank < a.topk) {
      picks.id[rank] = (int)c.y;
      picks.logit[rank] = key_value(c.x, 0.0f);  // where the choice is by logits
    }
    if (scored) {
      if (lane < n) picks.ranked[rank] = c;
      __syncwarp();
      uint2 p{}, q{};
      bool near = false;
      if (lane + 1 < n) {
        p = picks.ranked[lane], q = picks.ranked[lane + 1];
        const float v = key_value(p.x, 0.0f);
        near = v - key_value(q.x, 0.0f) <= bound(v);
      }
      const unsigned nears = __ballot_sync(kFull, near);
      if (nears & ((2u << (a.topk - 1)) - 1u)) {
        // Equal logits and biases are equal in any arithmetic.  The order counts up to the
        // topk-th candidate and through those that are the same as it: what is near to
        // one of them may stand before all of them.
        const bool same = near && p.x == q.x && row[p.y] == row[q.y] && a.bias[p.y] == a.bias[q.y];
        const unsigned sames = __ballot_sync(kFull, same);
        const int last = a.topk - 2 + __ffs(~(sames >> (a.topk - 1)));
        if (nears & ~sames & ((2u << last) - 1u))
          rank_exactly<T>(a, row, scores_exactly<T>(a, row, lmax), n, picks);
      }
    }
    __syncwarp();
    return;
  }

  // Otherwise (many equal values, or topk near 32) topk times the best key of the
  // warp; the lane whose expert was taken looks again.
  if (scored) {
    pick_exactly<T, EPL>(a, row, scores_exactly<T>(a, row, lmax), a.groups > 1 ? mask : 0xffffffffu, picks);
    return;
  }
#pragma unroll 1
  for (int s = 0; s < a.topk; ++s) {
    const uint32_t top = warp_max_key(best);
    if (top <= kNone) break;
    if (lane == __ffs(__ballot_sync(kFull, best == top)) - 1) {
      best = 0;
      int taken = -1;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        if (taken < 0 && key[j] == top) {
          taken = j;
          key[j] = 0;
          picks.logit[s] = l[j];
        }
        best = key[j] > best ? key[j] : best;
      }
      picks.id[s] = e0 + taken;
    }
  }
  __syncwarp();
}

}  // namespace

template <typename T, int EPL>
__global__ void __launch_bounds__(32 * kMaxWarps, EPL <= 8 ? 8 : EPL == 16 ? 6 : 4) route_topk_kernel(const RouteArgs a) {
  __shared__ Picks s_picks[kMaxWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.M) return;
  const T* row = static_cast<const T*>(a.logits) + (uint64_t)t * a.ld;
  Picks& picks = s_picks[threadIdx.x >> 5];

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
  select_experts<T, EPL>(a, row, l, lmax, zinv, picks);

  // Weights.  Renormalised ones are formed relative to the largest chosen
  // logit, so they are never 0 / 0: softmax exp(l - top); sigmoid
  // exp(l - base) / (1 + exp(l)) with base = min(0, top).  In FP32: a difference, one or
  // two exponentials and quotients of at most 2 ulp, the sum and two products; the
  // weights scale FP32 expert outputs, which carry larger errors.
  const int id = picks.id[lane];
  float x = -INFINITY;
  if (id >= 0) x = a.bias == nullptr ? picks.logit[lane] : clean_logit(logit_f32<T>(__ldg(row + id)));
  float base = a.softmax ? lmax : 0.0f;
  if (a.renorm) {
    base = key_value(__reduce_max_sync(kFull, order_key(x)), 0.0f);
    if (!a.softmax) base = fminf(base, 0.0f);
  }
  float w = 0.0f;
  if (id >= 0) {
    if (a.softmax) {
      w = expf(x - base);
    } else if (base < 0.0f) {
      w = __fdividef(expf(x - base), 1.0f + expf(x));
    } else {
      const float t = expf(-fabsf(x));
      w = __fdividef(x > 0.0f ? 1.0f : t, 1.0f + t);
    }
  }
  float norm = a.softmax ? zinv : 1.0f;
  if (a.renorm) {
    float sum = w;  // of lanes 0 .. topk - 1, the others' weights are 0
#pragma unroll 1
    for (int o = 1; o < a.topk; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
    norm = __fdividef(1.0f, sum);
  }
  if (lane < a.topk) {
    const uint64_t at = (uint64_t)t * a.topk + lane;
    a.ids[at] = id;
    a.weights[at] = id >= 0 ? w * norm * a.scale : 0.0f;
  }
}

namespace {

template <typename T>
cudaError_t launch_route_topk_of(const RouteArgs& a, cudaStream_t stream) {
  // One warp per CTA while that leaves every SM at most four tokens, one for each of its
  // schedulers; four for larger batches.
  const int warps = a.M <= 4u * (uint32_t)sm_count() ? 1 : kMaxWarps;
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
  a.vec_bias = r.num_experts % 32 == 0 && (a.per_lane & (a.per_lane - 1)) == 0 &&
               reinterpret_cast<uintptr_t>(r.bias) % (a.per_lane < 4 ? 4 * a.per_lane : 16) == 0;
  a.softmax = r.softmax;
  a.renorm = r.renormalize;
  a.scale = r.scale;
  return logits_f32 ? launch_route_topk_of<float>(a, stream) : launch_route_topk_of<uint16_t>(a, stream);
}

}  // namespace nvm
