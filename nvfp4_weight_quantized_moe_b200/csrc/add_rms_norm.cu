// Root-mean-square norm with the residual's addition and an output in BF16, in
// 8 bits with one scale per row, or both.
//
//   r = x + residual;  residual_out = r in the residual's type
//   y = r * rsqrt(mean(r^2) + eps) * weight;  out = bf16(y)
//   scale = max|y| / Q, q = y / scale rounded to nearest even (Q = 127 for int8,
//   448 for E4M3)
//
// The sum, the mean square and y are FP32, from r before its rounding to BF16, and
// out is y rounded once.  Since y is
// r * weight times one factor per row, q = r * weight * (Q / max|r * weight|):
// max and mean square are reduced together, in one pass over a row that stays in
// registers.  Roundings before a code's: r, the product, the quotient of the row
// and its product, as many as in dividing y by the scale; keeping the errors until
// the code is formed costs 2 us of 4 at 256 x 7168 (60 operations an element instead
// of 25) and moves one code in a million (int8 rows of 4096 with BF16 residual: 42 of
// 39 million off the 64-bit code, 51 with the division in FP32).
//
// Bound by HBM: each input is read once, each output written once (8192 x 4096
// BF16 with residual: 42.9 us, 96 % of the copy bandwidth).  A row belongs to one
// warp or one CTA; each thread moves 16 bytes per load where the pointers and
// strides allow it, single elements where they do not.

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace nvm {

namespace {

struct NormArgs {
  const void* x;
  const void* res;
  void* res_out;
  const void* weight;
  uint16_t* out;
  void* q;
  float* q_scale;
  uint64_t ldx, ldr;
  uint32_t rows;
  int hidden;
  int weight_f32;
  int q_kind;  // kQuantNone, kQuantInt8, kQuantE4M3
  float eps;
};

struct NoResidual {};

// VEC consecutive elements as loaded: floats or BF16 bits.
template <typename T, int VEC>
struct Raw {
  T v[VEC];
};
template <>
struct alignas(16) Raw<uint16_t, 8> {
  uint4 u;
};
template <>
struct alignas(16) Raw<float, 8> {
  uint4 u[2];
};

template <int VEC>
NVM_DEV void load_raw(Raw<uint16_t, VEC>& r, const uint16_t* p) {
  if constexpr (VEC == 8) r.u = *reinterpret_cast<const uint4*>(p);
  else r.v[0] = *p;
}
template <int VEC>
NVM_DEV void load_raw(Raw<float, VEC>& r, const float* p) {
  if constexpr (VEC == 8) {
    r.u[0] = reinterpret_cast<const uint4*>(p)[0];
    r.u[1] = reinterpret_cast<const uint4*>(p)[1];
  } else {
    r.v[0] = *p;
  }
}
NVM_DEV void unpack_bf16x8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <int VEC>
NVM_DEV void to_float(const Raw<uint16_t, VEC>& r, float (&f)[VEC]) {
  if constexpr (VEC == 8) unpack_bf16x8(r.u, f);
  else f[0] = bf16_bits_to_f32(r.v[0]);
}
template <int VEC>
NVM_DEV void to_float(const Raw<float, VEC>& r, float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    const uint32_t w[8] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w, r.u[1].x, r.u[1].y, r.u[1].z, r.u[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  } else {
    f[0] = r.v[0];
  }
}

NVM_DEV uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <int VEC>
NVM_DEV void store(uint16_t* p, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]),
                                              bf16x2_bits(f[4], f[5]), bf16x2_bits(f[6], f[7]));
  } else {
    const __nv_bfloat16 b = __float2bfloat16_rn(f[0]);
    *p = *reinterpret_cast<const uint16_t*>(&b);
  }
}
template <int VEC>
NVM_DEV void store(float* p, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *p = f[0];
  }
}

// Two values to E4M3 codes, nearest even, saturating at 448; NaN stays NaN.
NVM_DEV uint32_t e4m3x2_bits(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// What turns r * weight into the value that its code is nearest to: Q / the largest
// |r * weight|.  Values below 2^-60, whose quotient would leave FP32, are brought
// up by `lift` first (exact); a row of zeros gives zeros.
struct Step {
  float lift, step;
};
NVM_DEV Step code_step(float most, float range) {
  Step s{most < 0x1p-60f ? 0x1p64f : 1.0f, 0.0f};
  if (most > 0.0f) s.step = range / (most * s.lift);
  return s;
}

// Codes of VEC values.
template <int VEC>
NVM_DEV void store_codes(uint8_t* p, const float (&f)[VEC], int kind) {
  uint32_t word[(VEC + 3) / 4];
  if (kind == kQuantInt8) {
    // Adding 1.5 * 2^23 rounds to a whole number, whose low byte is the code.
    uint32_t c[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) c[j] = __float_as_uint(f[j] + 12582912.0f);
    if constexpr (VEC == 1) {
      word[0] = c[0];
    } else {
#pragma unroll
      for (int j = 0; j < VEC; j += 4)
        word[j / 4] = __byte_perm(__byte_perm(c[j], c[j + 1], 0x0040), __byte_perm(c[j + 2], c[j + 3], 0x0040), 0x5410);
    }
  } else if constexpr (VEC == 1) {
    word[0] = e4m3x2_bits(f[0], 0.0f);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; j += 4) word[j / 4] = e4m3x2_bits(f[j], f[j + 1]) | e4m3x2_bits(f[j + 2], f[j + 3]) << 16;
  }
  if constexpr (VEC == 8) *reinterpret_cast<uint2*>(p) = make_uint2(word[0], word[1]);
  else *p = (uint8_t)word[0];
}

// VEC weights from `at` on.  Not `whole`: between pieces, so the pieces on either
// side are loaded and shifted by at % 8 elements in three steps (two of 4 for
// FP32); where those pass the end of the row, single elements are.
template <int VEC>
NVM_DEV void load_weights(const NormArgs& a, int at, bool whole, float (&w)[VEC]) {
  if (a.weight_f32) {
    const float* p = static_cast<const float*>(a.weight) + at;
    if (whole) {
      Raw<float, VEC> r;
      load_raw(r, p);
      to_float(r, w);
      return;
    }
    if constexpr (VEC == 8) {
      const int s = at & 3;
      if (at - s + 12 <= a.hidden) {
        float f[12];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(p - s) + i);
          f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 10; ++i) f[i] = s & 2 ? f[i + 2] : f[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = s & 1 ? f[i + 1] : f[i];
        return;
      }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[j] = __ldg(p + j);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.weight) + at;
    if (whole) {
      Raw<uint16_t, VEC> r;
      load_raw(r, p);
      to_float(r, w);
      return;
    }
    if constexpr (VEC == 8) {
      const int s = at & 7;
      if (at - s + 16 <= a.hidden) {
        const uint4 lo = __ldg(reinterpret_cast<const uint4*>(p - s)), hi = __ldg(reinterpret_cast<const uint4*>(p - s) + 1);
        unpack_bf16x8(shift_u16x8(lo, hi, s), w);
        return;
      }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[j] = bf16_bits_to_f32(__ldg(p + j));
  }
}

// r of VEC elements.
template <typename XT, typename RT, typename RTs, int VEC>
NVM_DEV void add(const Raw<XT, VEC>& rx, const Raw<RTs, VEC>& rr, float (&r)[VEC]) {
  to_float(rx, r);
  if constexpr (!std::is_same<RT, NoResidual>::value) {
    float f[VEC];
    to_float(rr, f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[j] += f[j];
  }
}

// First pass over VEC elements: r to residual_out, its squares into `sum` and,
// for codes, the largest |r * weight| into `most`.
template <typename XT, typename RT, typename RTs, int VEC, bool CODES>
NVM_DEV void take(const NormArgs& a, uint64_t row, int at, const Raw<XT, VEC>& rx, const Raw<RTs, VEC>& rr,
                  const float (&w)[VEC], float& sum, float& most) {
  float r[VEC];
  add<XT, RT>(rx, rr, r);
  if (!std::is_same<RT, NoResidual>::value && a.res_out != nullptr)
    store<VEC>(static_cast<RTs*>(a.res_out) + row * (uint64_t)a.hidden + at, r);
#pragma unroll
  for (int j = 0; j < VEC; ++j) sum = fmaf(r[j], r[j], sum);
  if constexpr (CODES) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) most = fmaxf(most, fabsf(r[j] * w[j]));
  }
}

// Second pass: the codes and the norm.
template <typename XT, typename RT, typename RTs, int VEC, bool CODES>
NVM_DEV void give(const NormArgs& a, uint64_t row, int at, const Raw<XT, VEC>& rx, const Raw<RTs, VEC>& rr,
                  const float (&w)[VEC], const Step& step, float inv) {
  const uint64_t o = row * (uint64_t)a.hidden + at;
  float r[VEC];
  add<XT, RT>(rx, rr, r);
#pragma unroll
  for (int j = 0; j < VEC; ++j) r[j] *= w[j];
  if constexpr (CODES) {
    float c[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) c[j] = r[j] * step.lift * step.step;
    store_codes<VEC>(static_cast<uint8_t*>(a.q) + o, c, a.q_kind);
  }
  if (a.out != nullptr) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[j] *= inv;
    store<VEC>(a.out + o, r);
  }
}

}  // namespace

// blockDim = (threads per row, rows per CTA); threads per row is a multiple of
// 32, and 32 whenever a CTA holds more than one row.  A thread holds NV pieces
// of VEC elements, blockDim.x pieces apart, as they were loaded: r is formed again
// in the second pass, which keeps a piece in 4 to 16 registers and many rows on
// their way.  Pieces of 8 lie on multiples of 8 elements of the tensors; with ENDS
// a row that does not begin or end on one has up to 7 single elements at either
// end, one each for the first threads.
template <typename XT, typename RT, int VEC, int NV, bool ENDS, bool CODES>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const NormArgs a) {
  constexpr bool kRes = !std::is_same<RT, NoResidual>::value;
  using RTs = typename std::conditional<kRes, RT, uint16_t>::type;
  __shared__ float part_sum[32];
  __shared__ float part_most[32];
  griddep_wait();
  griddep_launch_dependents();
  const uint64_t row = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;  // whole warps: a row's threads leave together
  const int H = a.hidden, tid = (int)threadIdx.x;
  const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
  const RTs* res = static_cast<const RTs*>(a.res) + row * a.ldr;
  int head = 0, body = H, single = H;  // elements before the pieces and in them; this thread's single one
  if constexpr (ENDS) {
    head = min(H, (int)((0 - row * (uint64_t)H) & (VEC - 1)));
    body = (H - head) & ~(VEC - 1);
    single = tid >= 2 * VEC ? H : tid < head ? tid : tid + body;
  }
  const bool whole = !ENDS || head == 0;
  const bool lone = ENDS && single < H;

  Raw<XT, VEC> rx[NV];
  Raw<RTs, VEC> rr[NV];
  Raw<XT, 1> lx;
  Raw<RTs, 1> lr;
  float w[VEC], lw[1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * (int)blockDim.x + tid) * VEC;
    if (at < body) {
      load_raw(rx[i], x + head + at);
      if constexpr (kRes) load_raw(rr[i], res + head + at);
    }
  }
  if (lone) {
    load_raw(lx, x + single);
    if constexpr (kRes) load_raw(lr, res + single);
    load_weights<1>(a, single, true, lw);
  }
  // One piece per thread: its weights come with it.
  if (NV == 1 && tid * VEC < body) load_weights<VEC>(a, head + tid * VEC, whole, w);

  float sum = 0.0f;
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * (int)blockDim.x + tid) * VEC;
    if (at >= body) continue;
    if (NV > 1 && CODES) load_weights<VEC>(a, head + at, whole, w);
    take<XT, RT, RTs, VEC, CODES>(a, row, head + at, rx[i], rr[i], w, sum, most);
  }
  if (lone) take<XT, RT, RTs, 1, CODES>(a, row, single, lx, lr, lw, sum, most);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if constexpr (CODES) most = warp_max(most);
  if (blockDim.x > 32) {
    const int warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    if (lane == 0) {
      part_sum[warp] = sum;
      if constexpr (CODES) part_most[warp] = most;
    }
    __syncthreads();
    sum = lane < warps ? part_sum[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (CODES) most = warp_max(lane < warps ? part_most[lane] : 0.0f);
  }
  const float inv = rsqrtf(sum / (float)H + a.eps);
  const float range = a.q_kind == kQuantInt8 ? 127.0f : 448.0f;
  // Squares past the FP32 range make the row's factor and scale 0, and so its codes.
  const Step step = code_step(most, sum < INFINITY ? range : 0.0f);
  if (CODES && tid == 0) a.q_scale[row] = most * inv / range;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * (int)blockDim.x + tid) * VEC;
    if (at >= body) continue;
    if (NV > 1) load_weights<VEC>(a, head + at, whole, w);
    give<XT, RT, RTs, VEC, CODES>(a, row, head + at, rx[i], rr[i], w, step, inv);
  }
  if (lone) give<XT, RT, RTs, 1, CODES>(a, row, single, lx, lr, lw, step, inv);
}

namespace {

template <typename XT, typename RT, int VEC, bool ENDS, bool CODES>
cudaError_t launch_norm_of(const NormArgs& a, cudaStream_t stream) {
  const int pieces = (a.hidden + VEC - 1) / VEC;
  auto launch = [&](auto kernel, int nv) {
    const int tx = ((pieces + nv - 1) / nv + 31) / 32 * 32, ty = tx == 32 ? 4 : 1;
    return launch_pdl(kernel, dim3((a.rows + (uint32_t)ty - 1) / (uint32_t)ty), dim3(tx, ty), 0, stream, a);
  };
  if constexpr (VEC == 1) {
    if (pieces > 4096) return launch(add_rms_norm_kernel<XT, RT, VEC, 32, false, CODES>, 32);
    if (pieces > 1024) return launch(add_rms_norm_kernel<XT, RT, VEC, 4, false, CODES>, 4);
    return launch(add_rms_norm_kernel<XT, RT, VEC, 1, false, CODES>, 1);
  } else {
    // Up to a row per SM, one piece per thread: the shortest way through a row
    // (1 x 2048: 1.6 us, with two pieces 2.0).  More rows: fewer threads with more
    // bytes each, so that more rows are on their way per SM (one, two, four pieces:
    // 256 x 4096 BF16 3.2, 2.8, 3.6 us; 8192 x 4096 51.7, 45.0, 42.9; 8192 x 2048
    // 25.4, 22.7, 23.5; with FP32 in and residual 88, 76, 139).
    constexpr bool kNarrow = sizeof(XT) == 2 && !std::is_same<RT, float>::value;
    const uint32_t sms = (uint32_t)sm_count();
    int nv = 1;
    if (a.rows > sms && pieces > 32) nv = kNarrow && pieces >= 512 && a.rows > 8 * sms ? 4 : 2;
    if (pieces > 1024 * nv) nv = pieces > 2048 ? 4 : 2;
    if (nv == 4) return launch(add_rms_norm_kernel<XT, RT, VEC, 4, ENDS, CODES>, 4);
    if (nv == 2) return launch(add_rms_norm_kernel<XT, RT, VEC, 2, ENDS, CODES>, 2);
    return launch(add_rms_norm_kernel<XT, RT, VEC, 1, ENDS, CODES>, 1);
  }
}

template <typename XT, typename RT, bool CODES>
cudaError_t launch_norm_vec(const NormArgs& a, bool vec, cudaStream_t stream) {
  if (!vec) return launch_norm_of<XT, RT, 1, false, CODES>(a, stream);
  return a.hidden % 8 == 0 ? launch_norm_of<XT, RT, 8, false, CODES>(a, stream)
                           : launch_norm_of<XT, RT, 8, true, CODES>(a, stream);
}

template <typename XT, typename RT>
cudaError_t launch_norm_codes(const NormArgs& a, bool vec, cudaStream_t stream) {
  return a.q_kind != kQuantNone ? launch_norm_vec<XT, RT, true>(a, vec, stream)
                                : launch_norm_vec<XT, RT, false>(a, vec, stream);
}

template <typename XT>
cudaError_t launch_norm_res(const NormArgs& a, int res, bool vec, cudaStream_t stream) {
  if (a.res == nullptr) return launch_norm_codes<XT, NoResidual>(a, vec, stream);
  return res ? launch_norm_codes<XT, float>(a, vec, stream) : launch_norm_codes<XT, uint16_t>(a, vec, stream);
}

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

}  // namespace

cudaError_t launch_add_rms_norm(const NormConfig& c, cudaStream_t stream) {
  NormArgs a{};
  a.x = c.x;
  a.res = c.residual;
  a.res_out = c.residual_out;
  a.weight = c.weight;
  a.out = c.out;
  a.q = c.q;
  a.q_scale = c.q_scale;
  a.ldx = c.ldx;
  a.ldr = c.ldr;
  a.rows = c.rows;
  a.hidden = (int)c.hidden;
  a.weight_f32 = c.weight_f32;
  a.q_kind = c.q != nullptr ? c.q_kind : kQuantNone;
  a.eps = c.eps;
  // Pieces of 8 elements need every tensor to begin on 16 bytes (the codes on 8)
  // and every row to begin at the same place between pieces in all of them: the
  // outputs' rows are hidden apart.
  const bool vec = aligned(c.x, 16) && aligned(c.residual, 16) && aligned(c.residual_out, 16) &&
                   aligned(c.weight, 16) && aligned(c.out, 16) && aligned(c.q, 8) &&
                   c.ldx % 8 == c.hidden % 8 && (c.residual == nullptr || c.ldr % 8 == c.hidden % 8);
  return c.x_f32 ? launch_norm_res<float>(a, c.residual_f32, vec, stream)
                 : launch_norm_res<uint16_t>(a, c.residual_f32, vec, stream);
}

}  // namespace nvm
