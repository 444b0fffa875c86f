// Product of 8-bit integer matrices with a scale per token and per channel:
//
//   out[m, n] = x_scale[m] * w_scale[n] * sum_k x[m, k] w[n, k]  (+ bias[n])
//
// The sums are exact in 32-bit integers (K is bounded so that they cannot
// overflow), so every split of K gives the same bits; the sum, the two products
// with the scales and the addition of the bias are rounded to FP32 each
// (int8_scaled, the same in all kernels), then the result to the output's type.
//
// Small batches take the register-fed kernel of this file, larger ones the
// tensor-core kernels of int8_matmul_tc.cu (launch_int8_matmul has the rule).
//
// Register-fed kernel: one CTA per 16 channels and 8 TT tokens; its 4 or 8 warps
// split K in chunks of 64 and add their sums in shared memory.  mma.m16n8k32 (s8)
// takes the channels as rows and the tokens as columns.  A lane loads 16
// consecutive bytes of a row where the instruction wants four runs of four: the
// k order inside a chunk is permuted, identically for both operands, which a sum
// does not notice.  Bound by the weights' way from memory: 1 x 4096 x 2048 (tokens, n, k)
// 2.7 us with its 8.4 MB of weights in the L2 and 3.5 from HBM (1.3 us are the launch),
// 1 x 5120 x 4096 4.9 and 7.3: 16 rows of 64 bytes per load instruction, at most 98 KB in
// flight per SM.

#include <cmath>

#include "common.cuh"
#include "int8_epilogue.cuh"
#include "kernels.h"

namespace nvm {

namespace {

constexpr int kRegRows = 16;

NVM_DEV void mma_s8_16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

NVM_DEV void store_out(void* out, bool f32, uint64_t at, float v) {
  if (f32) {
    static_cast<float*>(out)[at] = v;
  } else {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    static_cast<uint16_t*>(out)[at] = *reinterpret_cast<const uint16_t*>(&b);
  }
}

}  // namespace

// WARPS split K; each has AHEAD chunks in flight, twice.
template <int TT, int WARPS, int AHEAD>
__global__ void __launch_bounds__(32 * WARPS) int8_matmul_reg_kernel(const Int8MatmulArgs a) {
  __shared__ int part[WARPS][8 * TT][kRegRows + 1];
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
  // The next AHEAD chunks are on their way while these are multiplied: a weight
  // byte takes about a microsecond to arrive.
  struct Chunk {
    uint4 u, v, b[TT];
  };
  Chunk now[AHEAD], next[AHEAD];
  auto load = [&](Chunk (&chunk)[AHEAD], int k0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int k = k0 + 64 * WARPS * i;
      const bool in = k + 16 * c < K;
      chunk[i].u = in && r0 ? ld_stream_v4(w0 + k) : zero;
      chunk[i].v = in && r1 ? ld_stream_v4(w1 + k) : zero;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t m = m0 + 8 * t + g;
        chunk[i].b[t] = zero;
        if (in && m < a.M)
          chunk[i].b[t] =
              __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.x) + (uint64_t)m * a.ldx + k + 16 * c));
      }
    }
  };
  constexpr int kStep = 64 * WARPS * AHEAD;
  load(now, 64 * warp);
  for (int k0 = 64 * warp; k0 < K; k0 += kStep) {
    if (k0 + kStep < K) load(next, k0 + kStep);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        mma_s8_16832(d[t], now[i].u.x, now[i].v.x, now[i].u.y, now[i].v.y, now[i].b[t].x, now[i].b[t].y);
        mma_s8_16832(d[t], now[i].u.z, now[i].v.z, now[i].u.w, now[i].v.w, now[i].b[t].z, now[i].b[t].w);
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) now[i] = next[i];
  }
  // d[t] holds channels g and g + 8 of tokens 8 t + 2 c, + 1.
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][8 * t + 2 * c + (i & 1)][g + 8 * (i >> 1)] = d[t][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * TT * kRegRows; i += 32 * WARPS) {
    const uint32_t m = m0 + i / kRegRows, n = n0 + i % kRegRows;
    if (m >= a.M || n >= a.N) continue;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += part[w][i / kRegRows][i % kRegRows];
    float v = int8_scaled(sum, a.x_scale[m], a.w_scale[n]);
    if (a.bias != nullptr) v = int8_biased(v, a.bias[n]);
    store_out(a.out, a.out_f32, (uint64_t)m * a.ldo + n, v);
  }
}

namespace {

template <int TT, int WARPS, int AHEAD>
cudaError_t launch_reg_of(const Int8MatmulArgs& a, uint64_t blocks, cudaStream_t stream) {
  return launch_pdl(int8_matmul_reg_kernel<TT, WARPS, AHEAD>, dim3((unsigned)blocks), dim3(32 * WARPS), 0, stream, a);
}

uint64_t reg_blocks(uint32_t M, uint32_t N, uint32_t tiles) {
  return (uint64_t)((N + kRegRows - 1) / kRegRows) * ((M + 8 * tiles - 1) / (8 * tiles));
}

// A long K is a chain of round trips to memory: eight warps with as many chunks in
// flight as registers allow (1 token, n = k = 4096: 3.6 us, with four warps and one
// chunk 7.1; weights in the L2).  A short one, or more CTAs than keep every SM busy,
// is better off with small CTAs (246 x 336 x 192: 2.1 us against 4.0).
bool reg_deep(uint64_t blocks, uint32_t K, int sms) { return K >= 1024 && blocks <= 4ull * sms; }

template <int TT>
cudaError_t launch_reg(const Int8MatmulArgs& a, bool deep, cudaStream_t stream) {
  const uint64_t blocks = reg_blocks(a.M, a.N, TT);
  if (blocks > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  constexpr int kLong = TT == 1 ? 4 : 2;
  return deep ? launch_reg_of<TT, 8, kLong>(a, blocks, stream) : launch_reg_of<TT, 4, 1>(a, blocks, stream);
}

// Which kernel takes a product: the shortest of the estimated times below, in
// microseconds.  Their forms follow the kernels (rounds of CTAs, a pace per
// stage of K, bytes through the L2 at a rate, an epilogue); the numbers are a
// fit to 446 shapes of 1 to 8192 tokens, n 64 to 8192, k 128 to 8192, measured on
// B200 in all nine forms.  Over those shapes the choice is 1.2 % slower than the
// best form in the geometric mean; each of the nine is the best for some.  Three
// sets of weights took turns, so those under 40 MB came from the L2: for a few tokens
// with weights from HBM the estimates are low (1 x 5120 x 4096: 4.9 us, from HBM 7.3).
struct Form {
  int bn;       // 0: register-fed; 64, 128: tiles of so many channels; 256: CTA pairs
  uint32_t by;  // register-fed: 8-token tiles; tiles: CTAs that split K
};

double estimate(uint32_t M, uint32_t N, uint32_t K, Form f, int sms) {
  auto over = [](uint64_t x, uint64_t y) { return (double)((x + y - 1) / y); };
  const double stages = over(K, 128);
  if (f.bn == 0) {
    const uint64_t ctas = reg_blocks(M, N, f.by);
    const double bytes = (double)ctas * K * (16.0 + 8 * f.by);
    const bool deep = reg_deep(ctas, K, sms);
    if (f.by == 1) return 1.3 + (deep ? over(K, 2048) * 0.38 : 0.0) + bytes / 7.7e6;
    return 1.3 + (deep ? over(K, 1024) * 0.43 : over(K, 256) * 0.14) + bytes / 8.1e6;
  }
  // 128-byte lines that 128 bytes of a row lie in, on average: rows are K bytes apart.
  const uint32_t low = K & (0u - K);
  const double lines = 2.0 - (low < 128 ? low : 128) / 128.0;
  if (f.bn == 256)
    return 4.5 + std::ceil(over(M, 256) * over(N, 256) / (sms / 2)) * stages * 0.35 * (0.78 + 0.22 * lines);
  const double ctas = over(M, 128) * over(N, f.bn) * f.by, per_sm = std::ceil(ctas / int8_tile_slots(f.by));
  const double own = std::ceil(stages / f.by), rows = M < 128 ? over(M, 8) * 8 : 128;
  // A stage takes its products or its lines through the SM's copy engine; two CTAs of
  // an SM overlap.
  const double stage = std::fmax(f.bn == 64 ? 0.17 : 0.18, (rows + f.bn) * lines * 0.63e-3);
  const double pace = own * stage * (per_sm == 1 ? 1 : per_sm * 0.81);
  const double bytes = ctas * own * (rows + f.bn) * 128, through = bytes / 17e6 * (0.53 + 0.47 * lines);
  const double full = 0.5 + 0.5 * rows / 128;
  const double tail = f.by == 1 ? per_sm * (f.bn == 64 ? 0.75 : 2.8) * full : 1.7 + per_sm * (f.bn / 64) * full;
  return 2.1 + std::fmax(pace, through) + tail;
}

}  // namespace

Int8Form int8_form(uint32_t M, uint32_t N, uint32_t K) {
  static constexpr Form kForms[] = {{0, 1}, {0, 2}, {64, 1}, {64, 2}, {64, 4}, {64, 8}, {128, 1}, {128, 4}, {256, 1}};
  const int sms = sm_count();
  Form best = kForms[0];
  double least = estimate(M, N, K, best, sms);
  for (const Form& f : kForms) {
    if (f.bn > 0 && f.by > (K + 127) / 128) continue;  // a stage of K for each CTA at least
    const double t = estimate(M, N, K, f, sms);
    if (t < least) {
      least = t;
      best = f;
    }
  }
  if (best.bn == 0) return {(uint32_t)kRegRows, 8 * best.by, 1, reg_deep(reg_blocks(M, N, best.by), K, sms)};
  if (best.bn == 256) return {256, 256, 1, true};
  return {(uint32_t)best.bn, 128, best.by, int8_tile_deep(M, N, best.bn, best.by)};
}

cudaError_t launch_int8_matmul(const Int8MatmulArgs& a, cudaStream_t stream) {
  const Int8Form f = int8_form(a.M, a.N, a.K);
  if (f.channels == 256) return launch_int8_pair(a, stream);
  if (f.channels >= 64) return launch_int8_tile(a, f, stream);
  return f.tokens == 8 ? launch_reg<1>(a, f.deep, stream) : launch_reg<2>(a, f.deep, stream);
}

}  // namespace nvm
