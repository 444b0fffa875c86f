// Product of 8-bit integer matrices with a scale per token and per channel:
//
//   out[m, n] = x_scale[m] * w_scale[n] * sum_k x[m, k] w[n, k]  (+ bias[n])
//
// The sums are exact in 32-bit integers (K is bounded so that they cannot
// overflow), so every split of K gives the same bits; scales and bias are
// applied in FP32 and the result is rounded once to the output's type.
//
// Small batches take the register-fed kernel of this file, larger ones the
// tensor-core kernels of int8_matmul_tc.cu (launch_int8_matmul has the rule).
//
// Register-fed kernel: one CTA per 16 channels and 8 TT tokens; its warps split
// K in chunks of 64 and add their sums in shared memory.  mma.m16n8k32 (s8)
// takes the channels as rows and the tokens as columns.  A lane loads 16
// consecutive bytes of a row where the instruction wants four runs of four: the
// k order inside a chunk is permuted, identically for both operands, which a sum
// does not notice.

#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace nvm {

namespace {

constexpr int kRegWarps = 4;
constexpr int kRegRows = 16;

NVM_DEV void mma_s8_16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

NVM_DEV float scaled(int sum, float xs, float ws) { return (float)sum * xs * ws; }

NVM_DEV void store_out(void* out, bool f32, uint64_t at, float v) {
  if (f32) {
    static_cast<float*>(out)[at] = v;
  } else {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    static_cast<uint16_t*>(out)[at] = *reinterpret_cast<const uint16_t*>(&b);
  }
}

}  // namespace

template <int TT>
__global__ void __launch_bounds__(32 * kRegWarps) int8_matmul_reg_kernel(const Int8MatmulArgs a) {
  __shared__ int part[kRegWarps][8 * TT][kRegRows + 1];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t nblocks = (a.N + kRegRows - 1) / kRegRows;
  const uint32_t n0 = blockIdx.x % nblocks * kRegRows, m0 = blockIdx.x / nblocks * (8 * TT);
  const uint8_t* w0 = static_cast<const uint8_t*>(a.w) + (uint64_t)(n0 + g) * a.K + 16 * c;
  const uint8_t* w1 = w0 + (uint64_t)8 * a.K;
  const bool r0 = n0 + g < a.N, r1 = n0 + g + 8 < a.N;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  int d[TT][4] = {};
  const int K = (int)a.K;
#pragma unroll 2
  for (int k0 = 64 * warp; k0 < K; k0 += 64 * kRegWarps) {
    const bool in = k0 + 16 * c < K;
    const uint4 u = in && r0 ? ld_stream_v4(w0 + k0) : zero;
    const uint4 v = in && r1 ? ld_stream_v4(w1 + k0) : zero;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint32_t m = m0 + 8 * t + g;
      uint4 b = zero;
      if (in && m < a.M)
        b = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.x) + (uint64_t)m * a.ldx + k0 + 16 * c));
      mma_s8_16832(d[t], u.x, v.x, u.y, v.y, b.x, b.y);
      mma_s8_16832(d[t], u.z, v.z, u.w, v.w, b.z, b.w);
    }
  }
  // d[t] holds channels g and g + 8 of tokens 8 t + 2 c, + 1.
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][8 * t + 2 * c + (i & 1)][g + 8 * (i >> 1)] = d[t][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * TT * kRegRows; i += 32 * kRegWarps) {
    const uint32_t m = m0 + i / kRegRows, n = n0 + i % kRegRows;
    if (m >= a.M || n >= a.N) continue;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kRegWarps; ++w) sum += part[w][i / kRegRows][i % kRegRows];
    float v = scaled(sum, a.x_scale[m], a.w_scale[n]);
    if (a.bias != nullptr) v += a.bias[n];
    store_out(a.out, a.out_f32, (uint64_t)m * a.ldo + n, v);
  }
}

namespace {

template <int TT>
cudaError_t launch_reg(const Int8MatmulArgs& a, cudaStream_t stream) {
  const uint64_t blocks = (uint64_t)((a.N + kRegRows - 1) / kRegRows) * ((a.M + 8 * TT - 1) / (8 * TT));
  if (blocks > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  return launch_pdl(int8_matmul_reg_kernel<TT>, dim3((unsigned)blocks), dim3(32 * kRegWarps), 0, stream, a);
}

}  // namespace

namespace {

// Which kernel takes a product: the shortest of the estimated times below, in
// microseconds.  Their forms follow the kernels (rounds of CTAs, a pace per
// stage of K, bytes through the L2 at a rate, an epilogue); the numbers are a
// fit to 178 shapes of 1 to 8192 tokens, n 64 to 16384, k 128 to 8192, measured on
// B200 in all nine forms.  Over those shapes the choice is 1.3 % slower than the
// best form in the geometric mean, where any single kernel is over 40 %.
struct Form {
  int bn;       // 0: register-fed; 64, 128: tiles of so many channels; 256: CTA pairs
  uint32_t by;  // register-fed: 8-token tiles; tiles: CTAs that split K
};

double estimate(const Int8MatmulArgs& a, Form f, double sms) {
  auto over = [](uint64_t x, uint64_t y) { return (double)((x + y - 1) / y); };
  const double stages = over(a.K, 128);
  if (f.bn == 0) {
    const double ctas = over(a.N, 16) * over(a.M, 8 * f.by);
    const bool one = f.by == 1;
    return 1.1 + over(a.K, 256) * (one ? 0.29 : 0.44) + ctas * a.K * (16.0 + 8 * f.by) / (one ? 11e6 : 13e6);
  }
  if (f.bn == 256) return 5.1 + std::ceil(over(a.M, 256) * over(a.N, 256) / std::floor(sms / 2)) * stages * 0.39;
  const double ctas = over(a.M, 128) * over(a.N, f.bn) * f.by, per_sm = std::ceil(ctas / sms);
  const double own = std::ceil(stages / f.by), rows = a.M < 128 ? over(a.M, 8) * 8 : 128;
  const double pace = own * 0.43 * (per_sm == 1 ? 1 : per_sm * 0.59);  // two CTAs of an SM overlap
  const double bytes = ctas * own * (rows + f.bn) * 128 / 7.8e6;
  const double tail = f.by == 1 ? per_sm * (f.bn == 64 ? 0.63 : 2.8) : 2.4 + per_sm * 0.57 * (f.bn / 64);
  return 1.1 + (pace > bytes ? pace : bytes) + tail;
}

}  // namespace

cudaError_t launch_int8_matmul(const Int8MatmulArgs& a, cudaStream_t stream) {
  static constexpr Form kForms[] = {{0, 1}, {0, 2}, {64, 1}, {64, 2}, {64, 4}, {64, 8}, {128, 1}, {128, 4}, {256, 1}};
  const double sms = sm_count();
  Form best = kForms[0];
  double least = estimate(a, best, sms);
  for (const Form& f : kForms) {
    if (f.bn > 0 && f.by > (a.K + 127) / 128) continue;  // a stage of K for each CTA at least
    const double t = estimate(a, f, sms);
    if (t < least) {
      least = t;
      best = f;
    }
  }
  if (best.bn == 0) return best.by == 1 ? launch_reg<1>(a, stream) : launch_reg<2>(a, stream);
  if (best.bn == 256) return launch_int8_pair(a, stream);
  return launch_int8_tile(a, best.bn, best.by, stream);
}

}  // namespace nvm
