// Root-mean-square norm with the residual's addition and an output in BF16, in
// 8 bits with one scale per row, or both.
//
//   r = x + residual;  residual_out = r in the residual's type
//   y = r * rsqrt(mean(r^2) + eps) * weight;  out = bf16(y)
//   scale = max|y| / Q, q = y / scale rounded to nearest even (Q = 127 for int8,
//   448 for E4M3)
//
// The sum, the mean square and y are FP32, and out and q are rounded once from
// y: the residual's rounding to BF16 does not enter the norm.  Since y is
// r * weight times one factor per row, q = r * weight * (Q / max|r * weight|):
// max and mean square are reduced together, in one pass over a row that stays in
// registers.
//
// Bound by HBM: each input is read once, each output written once.  A row
// belongs to one warp (hidden up to 1024) or one CTA; each thread moves 16 bytes
// per load where the pointers, strides and hidden allow it, single elements
// where they do not.

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
// To int8, nearest even, within +-127; NaN gives 0.
NVM_DEV uint32_t int8_bits(float v) { return (uint32_t)__float2int_rn(fminf(fmaxf(v, -127.0f), 127.0f)) & 0xffu; }

template <int VEC>
NVM_DEV void store_codes(uint8_t* p, const float (&f)[VEC], int kind) {
  if constexpr (VEC == 8) {
    uint2 u;
    if (kind == kQuantInt8) {
      u.x = int8_bits(f[0]) | int8_bits(f[1]) << 8 | int8_bits(f[2]) << 16 | int8_bits(f[3]) << 24;
      u.y = int8_bits(f[4]) | int8_bits(f[5]) << 8 | int8_bits(f[6]) << 16 | int8_bits(f[7]) << 24;
    } else {
      u.x = e4m3x2_bits(f[0], f[1]) | e4m3x2_bits(f[2], f[3]) << 16;
      u.y = e4m3x2_bits(f[4], f[5]) | e4m3x2_bits(f[6], f[7]) << 16;
    }
    *reinterpret_cast<uint2*>(p) = u;
  } else {
    *p = (uint8_t)(kind == kQuantInt8 ? int8_bits(f[0]) : e4m3x2_bits(f[0], 0.0f) & 0xffu);
  }
}

}  // namespace

// blockDim = (threads per row, rows per CTA); threads per row is a multiple of
// 32, and 32 whenever a CTA holds more than one row.  A thread holds NV pieces
// of VEC elements, blockDim.x pieces apart.
template <typename XT, typename RT, int VEC, int NV>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const NormArgs a) {
  constexpr bool kRes = !std::is_same<RT, NoResidual>::value;
  using RTs = typename std::conditional<kRes, RT, uint16_t>::type;
  __shared__ float part_sum[32], part_max[32];
  griddep_wait();
  griddep_launch_dependents();
  const uint64_t row = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;  // whole warps: a row's threads leave together
  const int H = a.hidden;
  const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
  const RTs* res = static_cast<const RTs*>(a.res) + row * a.ldr;

  Raw<XT, VEC> rx[NV];
  Raw<RTs, VEC> rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * (int)blockDim.x + (int)threadIdx.x) * VEC;
    if (at < H) {
      load_raw(rx[i], x + at);
      if constexpr (kRes) load_raw(rr[i], res + at);
    }
  }
  // r, then r * weight; the mean square of the one, the largest of the other.
  float v[NV][VEC];
  float sum = 0.0f, most = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * (int)blockDim.x + (int)threadIdx.x) * VEC;
    if (at >= H) continue;
    float w[VEC];
    if (a.weight_f32) {
      Raw<float, VEC> rw;
      load_raw(rw, static_cast<const float*>(a.weight) + at);
      to_float(rw, w);
    } else {
      Raw<uint16_t, VEC> rw;
      load_raw(rw, static_cast<const uint16_t*>(a.weight) + at);
      to_float(rw, w);
    }
    to_float(rx[i], v[i]);
    if constexpr (kRes) {
      float f[VEC];
      to_float(rr[i], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] += f[j];
      if (a.res_out != nullptr) store<VEC>(static_cast<RTs*>(a.res_out) + row * (uint64_t)H + at, v[i]);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      sum = fmaf(v[i][j], v[i][j], sum);
      v[i][j] *= w[j];
      most = fmaxf(most, fabsf(v[i][j]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  most = warp_max(most);
  if (blockDim.x > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) {
      part_sum[warp] = sum;
      part_max[warp] = most;
    }
    __syncthreads();
    sum = lane < warps ? part_sum[lane] : 0.0f;
    most = lane < warps ? part_max[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = warp_max(most);
  }
  const float inv = rsqrtf(sum / (float)H + a.eps);
  const float range = a.q_kind == kQuantInt8 ? 127.0f : 448.0f;
  // Q / max|r * weight| leaves FP32 for a row of almost nothing: such values are
  // brought up by 2^64 first (exact), a row of zeros gives zeros.
  const float lift = most < 0x1p-60f ? 0x1p64f : 1.0f;
  const float step = most > 0.0f ? range / (most * lift) : 0.0f;
  if (a.q_kind != kQuantNone && threadIdx.x == 0) a.q_scale[row] = most * inv / range;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * (int)blockDim.x + (int)threadIdx.x) * VEC;
    if (at >= H) continue;
    const uint64_t o = row * (uint64_t)H + at;
    if (a.q_kind != kQuantNone) {
      float f[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = v[i][j] * lift * step;
      store_codes<VEC>(static_cast<uint8_t*>(a.q) + o, f, a.q_kind);
    }
    if (a.out != nullptr) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] *= inv;
      store<VEC>(a.out + o, v[i]);
    }
  }
}

namespace {

template <typename XT, typename RT, int VEC>
cudaError_t launch_norm_of(const NormArgs& a, cudaStream_t stream) {
  const int pieces = (a.hidden + VEC - 1) / VEC;
  const int nv = pieces > 2048 ? 4 : pieces > 1024 ? 2 : 1;
  int tx = ((pieces + nv - 1) / nv + 31) / 32 * 32;
  const int ty = tx == 32 ? 4 : 1;
  const dim3 block(tx, ty), grid((unsigned)((a.rows + (uint32_t)ty - 1) / (uint32_t)ty));
  if constexpr (VEC == 1) {
    if (nv == 4 && pieces > 4096) {
      tx = ((pieces + 31) / 32 + 31) / 32 * 32;
      return launch_pdl(add_rms_norm_kernel<XT, RT, VEC, 32>, grid, dim3(tx, 1), 0, stream, a);
    }
  }
  if (nv == 4) return launch_pdl(add_rms_norm_kernel<XT, RT, VEC, 4>, grid, block, 0, stream, a);
  if (nv == 2) return launch_pdl(add_rms_norm_kernel<XT, RT, VEC, 2>, grid, block, 0, stream, a);
  return launch_pdl(add_rms_norm_kernel<XT, RT, VEC, 1>, grid, block, 0, stream, a);
}

template <typename XT, typename RT>
cudaError_t launch_norm_vec(const NormArgs& a, bool vec, cudaStream_t stream) {
  return vec ? launch_norm_of<XT, RT, 8>(a, stream) : launch_norm_of<XT, RT, 1>(a, stream);
}

template <typename XT>
cudaError_t launch_norm_res(const NormArgs& a, int res, bool vec, cudaStream_t stream) {
  if (a.res == nullptr) return launch_norm_vec<XT, NoResidual>(a, vec, stream);
  return res ? launch_norm_vec<XT, float>(a, vec, stream) : launch_norm_vec<XT, uint16_t>(a, vec, stream);
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
  // 16-byte pieces need every pointer on 16 bytes (the codes' on 8) and whole
  // pieces per row; row strides that keep the rows there (8 BF16, 4 FP32).
  const bool vec = c.hidden % 8 == 0 && aligned(c.x, 16) && aligned(c.residual, 16) &&
                   aligned(c.residual_out, 16) && aligned(c.weight, 16) && aligned(c.out, 16) &&
                   aligned(c.q, 8) && c.ldx % (c.x_f32 ? 4 : 8) == 0 &&
                   c.ldr % (c.residual_f32 ? 4 : 8) == 0;
  return c.x_f32 ? launch_norm_res<float>(a, c.residual_f32, vec, stream)
                 : launch_norm_res<uint16_t>(a, c.residual_f32, vec, stream);
}

}  // namespace nvm
