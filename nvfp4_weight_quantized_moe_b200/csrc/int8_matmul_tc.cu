// The int8 product on the tensor cores (tcgen05.mma.kind::i8), for batches of
// more tokens than the register-fed kernel takes; see int8_matmul.cu for the
// operator.  Tokens are the M side of the instruction, channels the N side, so a
// thread of the epilogue holds one token's sums.  Operand tiles come by TMA as
// 128-byte rows with 128-byte swizzle; what lies past M, N or K reads as zero
// and adds nothing.
//
// int8_tile_kernel: one CTA per 128 x BN tile, and, where the tiles alone would
// leave SMs idle, a cluster of S CTAs per tile that splits K.  Each CTA of the
// cluster leaves its sums in shared memory; CTA r adds rows 128 r / S ... of all
// of them through distributed shared memory and writes them out.  Integer sums:
// the same bits for every S.
//
// int8_pair_kernel: persistent over 256 x 256 tiles, one CTA pair
// (tcgen05.mma.cta_group::2) per two SMs: each CTA holds 128 token rows and
// loads half of the channels' rows, so an SM reads 32 KB of shared memory per
// 128 k of a 256 x 256 tile and the operands' L2 traffic is half that of 128 x
// 128 tiles.  Two 256-column accumulators fill tensor memory, so a tile's
// epilogue overlaps the next tile's products.  Warp 0 loads, warp 1 of the
// first CTA issues, warps 2-9 drain (two per TMEM lane quarter, half of the
// columns each).
//
// Measured: 8192 x 8192 x 4096 (tokens, n, k) 169 us, 3.25 * 10^15 operations a second,
// 99 % of twice the measured BF16 rate.  Below k of about 1000 the outputs bound it: 3 us
// per round of tiles.  Tiles: 256 x 2048 x 7168 in 128 CTAs 9.0 us, of which 5 are launch,
// cluster exchange and epilogue, the rest the operands' way from the L2.
//
// Every wait is bounded; on timeout a CTA flags the device error word and skips
// its remaining waits.

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "int8_epilogue.cuh"
#include "kernels.h"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace nvm {

namespace {

constexpr int kStageK = 128;   // bytes of K per stage: one swizzled row
constexpr int kTileM = 128;

NVM_DEV uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// The outputs of one warp's 32 token rows (lane = row, from TMEM at `taddr`) and
// `cols` columns, written along the rows: each lane packs its row in pieces of
// 16 bytes, which go through 4 KB of shared memory (128 bytes per row, piece p of
// row r at p ^ (r % 8): no bank conflicts either way) so that 8 lanes write 128
// consecutive bytes.  ws and bias are the columns' in shared memory.  Rows
// from M on and columns from N on are not written.
template <bool F32>
NVM_DEV void drain_rows(uint32_t taddr, int cols, uint8_t* stage, const float* ws, const float* bias, float xs,
                        const Int8MatmulArgs& a, uint32_t m0, uint32_t n0) {
  constexpr int kPer = F32 ? 4 : 8;    // outputs per piece
  constexpr int kChunk = 8 * kPer;     // columns per pass
  if (m0 >= a.M) return;  // a warp without rows
  const int lane = threadIdx.x & 31, rows = a.M - m0 < 32u ? (int)(a.M - m0) : 32;
  const uint64_t elem = F32 ? 4 : 2;
  const bool vec = a.ldo * elem % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
#pragma unroll 1
  for (int c0 = 0; c0 < cols && n0 + c0 < a.N; c0 += kChunk) {
#pragma unroll
    for (int h = 0; h < kChunk / 32; ++h) {
      uint32_t d[32];
      tmem_ld32(taddr + c0 + 32 * h, d);
      tmem_wait_ld();
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 w4 = *reinterpret_cast<const float4*>(ws + c0 + 32 * h + j);
        v[j] = int8_scaled((int)d[j], xs, w4.x);
        v[j + 1] = int8_scaled((int)d[j + 1], xs, w4.y);
        v[j + 2] = int8_scaled((int)d[j + 2], xs, w4.z);
        v[j + 3] = int8_scaled((int)d[j + 3], xs, w4.w);
      }
      if (a.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = int8_biased(v[j], bias[c0 + 32 * h + j]);
      }
#pragma unroll
      for (int p = 0; p < 32 / kPer; ++p) {
        uint4 u;
        if constexpr (F32)
          u = make_uint4(__float_as_uint(v[4 * p]), __float_as_uint(v[4 * p + 1]), __float_as_uint(v[4 * p + 2]),
                         __float_as_uint(v[4 * p + 3]));
        else
          u = make_uint4(bf16_pair(v[8 * p], v[8 * p + 1]), bf16_pair(v[8 * p + 2], v[8 * p + 3]),
                         bf16_pair(v[8 * p + 4], v[8 * p + 5]), bf16_pair(v[8 * p + 6], v[8 * p + 7]));
        const int piece = h * (32 / kPer) + p;
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((piece ^ (lane & 7)) << 4)) = u;
      }
    }
    __syncwarp();
    if (vec && n0 + c0 + kChunk <= a.N) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 3), p = lane & 7;
        const uint4 u = *reinterpret_cast<const uint4*>(stage + r * 128 + ((p ^ (r & 7)) << 4));
        if (r < rows)
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + ((uint64_t)(m0 + r) * a.ldo + n0 + c0 + p * kPer) * elem) = u;
      }
    } else {
      // A row distance that is no whole number of pieces, or the last columns.
      const int left = (int)(a.N - (n0 + c0) < (uint32_t)kChunk ? a.N - (n0 + c0) : kChunk);
      if constexpr (F32) {
        float* out = static_cast<float*>(a.out) + (uint64_t)m0 * a.ldo + n0 + c0 + lane;
        if (lane < left) {
#pragma unroll 8
          for (int r = 0; r < rows; ++r, out += a.ldo)
            *out = *reinterpret_cast<const float*>(stage + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
        }
      } else {
        uint16_t* out = static_cast<uint16_t*>(a.out) + (uint64_t)m0 * a.ldo + n0 + c0;
        auto staged = [&](int r, int p) { return *reinterpret_cast<const uint4*>(stage + r * 128 + ((p ^ (r & 7)) << 4)); };
        auto value = [&](int r, int c) {
          return *reinterpret_cast<const uint16_t*>(stage + r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2);
        };
        if (left == kChunk) {
          // `head` elements before the row's first multiple of 16 bytes, 7 pieces
          // shifted together from the staged ones (8 where head is 0), the rest
          // behind them: one element each for the row's 8 lanes.
#pragma unroll 2
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3), p = lane & 7;
            if (r >= rows) continue;
            uint16_t* row = out + (uint64_t)r * a.ldo;
            const int head = (int)((0 - (reinterpret_cast<uintptr_t>(row) >> 1)) & 7);
            if (p < 7 || head == 0)
              *reinterpret_cast<uint4*>(row + head + 8 * p) = shift_u16x8(staged(r, p), staged(r, p < 7 ? p + 1 : p), head);
            if (head != 0) {
              const int c = p < head ? p : kChunk - 8 + p;
              row[c] = value(r, c);
            }
          }
        } else {
          for (int i = lane; i < rows * left; i += 32) {
            const int r = i / left, c = i % left;
            out[(uint64_t)r * a.ldo + c] = value(r, c);
          }
        }
      }
    }
    __syncwarp();
  }
}

NVM_DEV int4 ld_cluster_int4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// One lane of the warp, in a form from which the compiler sees that it is one.  The
// operands of copies and products live in the warp's uniform registers: with a whole
// warp that loops and one elected lane that issues they stay there, while behind
// `lane == 0` a product took 112 cycles to issue whatever its size (128 x 2048 x 8192 in
// 32 tiles: 18.1 us, elected 11.3; 8192 x 8192 x 4096 in pairs: 176 and 169).
NVM_DEV bool elect_one() {
  uint32_t v;
  asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(v));
  return v != 0;
}
NVM_DEV void tmap_prefetch(const void* tmap) { asm volatile("prefetch.tensormap [%0];" ::"l"(tmap) : "memory"); }

// DEEP: a ring that takes the SM, for grids of at most one CTA per SM.  With 64
// channels a barrier is for two stages of K: the four products of a stage take 0.07 us,
// less than the way from barrier to barrier (128 x 2048 x 8192 without a split: 12.8 us
// with one stage to a barrier, 11.3 with two; 128 channels 14.5 and 15.3).  Two CTAs of
// an SM hide each other's.
template <int BN, bool DEEP>
struct TileCfg {
  static constexpr int GROUP = DEEP && BN == 64 ? 2 : 1;      // stages to a barrier
  static constexpr int STAGES = BN == 64 ? 4 : DEEP ? 6 : 3;  // groups in the ring
  static constexpr int A_BYTES = kTileM * kStageK;
  static constexpr int B_BYTES = BN * kStageK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int GROUP_BYTES = GROUP * STAGE_BYTES;
  static constexpr int PITCH = BN + 4;  // ints between rows of the staged sums
  static constexpr int OFF_SCALE = STAGES * GROUP_BYTES;  // floats: tokens' [128], channels' [BN], biases [BN]
  static constexpr int OFF_BAR = OFF_SCALE + 4 * (kTileM + 2 * BN);
  // full[STAGES], empty[STAGES], done
  static constexpr int NBAR = 2 * STAGES + 1;
  static constexpr int OFF_TMEM = OFF_BAR + 8 * NBAR;
  static constexpr int OFF_ABORT = OFF_TMEM + 16;
  static constexpr int SMEM = OFF_ABORT + 16 + 1024;
  static_assert(kTileM * PITCH * 4 <= OFF_SCALE && 4 * 4096 <= OFF_SCALE, "staged sums and rows fit the ring");
  static_assert((DEEP ? 1 : 2) * (SMEM + 1024) <= 228 * 1024, "one or two CTAs per SM");
  // Two CTAs of this size are all an SM holds, with anything that shares it: no
  // allocation of tensor memory ever waits for another cluster's.
  static_assert((DEEP ? 2 : 3) * (SMEM + 1024) > 228 * 1024 && 2 * BN <= 512, "tensor memory");
  static_assert(tc_smem_safe(SMEM, BN), "no pairs of two kernels wait for each other's tensor memory");
};

constexpr int kTileThreads = 192;  // warp 0 loads, warp 1 issues, warps 2-5 drain

}  // namespace

template <int BN, bool DEEP>
__global__ void __launch_bounds__(kTileThreads)
    int8_tile_kernel(const Int8MatmulArgs a, const uint32_t split, const uint32_t x_rows,
                     const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w) {
  using C = TileCfg<BN, DEEP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t s_base = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (s_base - raw_base);
  const uint32_t full = s_base + C::OFF_BAR;
  const uint32_t empty = full + 8 * C::STAGES;
  const uint32_t done = empty + 8 * C::STAGES;
  float* scales = reinterpret_cast<float*>(smem + C::OFF_SCALE);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    tmap_prefetch(&tm_x);
    tmap_prefetch(&tm_w);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  const uint32_t rank = split > 1 ? cluster_ctarank() : 0;
  const uint32_t tiles_n = (a.N + BN - 1) / BN;
  const uint32_t tile = blockIdx.x / split;
  const uint32_t m0 = tile / tiles_n * kTileM, n0 = tile % tiles_n * BN;
  const uint32_t nst = (a.K + kStageK - 1) / kStageK;
  const uint32_t st_lo = (uint32_t)((uint64_t)nst * rank / split);
  const uint32_t st_hi = (uint32_t)((uint64_t)nst * (rank + 1) / split);

  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait(bar, parity)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp == 0) {
    const bool one = elect_one();
    uint32_t i = 0;
    for (uint32_t st = st_lo; st < st_hi; st += C::GROUP, ++i) {
      const uint32_t slot = i % C::STAGES, round = i / C::STAGES;
      if (round > 0 && !__all_sync(0xffffffffu, wait(empty + 8 * slot, (round - 1) & 1))) break;
      const uint32_t bar = full + 8 * slot, n = min((uint32_t)C::GROUP, st_hi - st);
      if (one) {
        mbar_arrive_expect_tx(bar, n * (x_rows * kStageK + C::B_BYTES));
        for (uint32_t g = 0; g < n; ++g) {
          const uint32_t dst = s_base + slot * C::GROUP_BYTES + g * C::STAGE_BYTES;
          tma_load_2d(dst, &tm_x, (int)((st + g) * kStageK), (int)m0, bar);
          tma_load_2d(dst + C::A_BYTES, &tm_w, (int)((st + g) * kStageK), (int)n0, bar);
        }
      }
      __syncwarp();
    }
    // Nothing may still land in this CTA's memory when it goes on.
    for (uint32_t j = i > (uint32_t)C::STAGES ? i - C::STAGES : 0; j < i; ++j)
      mbar_wait(full + 8 * (j % C::STAGES), (j / C::STAGES) & 1);
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_s8_s32(kTileM, BN);
    const bool one = elect_one();
    uint32_t i = 0;
    for (uint32_t st = st_lo; st < st_hi; st += C::GROUP, ++i) {
      const uint32_t slot = i % C::STAGES;
      if (!__all_sync(0xffffffffu, wait(full + 8 * slot, (i / C::STAGES) & 1))) break;
      tc_fence_after();
      if (one) {
#pragma unroll
        for (int g = 0; g < C::GROUP; ++g) {
          if (st + g >= st_hi) break;
          const uint32_t abase = s_base + slot * C::GROUP_BYTES + g * C::STAGE_BYTES, bbase = abase + C::A_BYTES;
#pragma unroll
          for (int k = 0; k < kStageK / 32; ++k)
            tc_mma_s8_ss(tmem, smem_desc_sw128(abase + 32 * k), smem_desc_sw128(bbase + 32 * k), idesc,
                         i > 0 || g > 0 || k > 0 ? 1u : 0u);
        }
        tc_commit(empty + 8 * slot);
      }
      __syncwarp();
    }
    if (one) tc_commit(done);
    __syncwarp();
    mbar_wait(done, 0);  // no MMA may still run when the tensor memory is freed
    __syncwarp();
  } else {
    const int q = warp & 3, row = 32 * q + lane;
    const int et = tid - 64;  // 0 .. 127
    scales[et] = m0 + et < a.M ? __ldg(a.x_scale + m0 + et) : 0.0f;
    for (int c = et; c < BN; c += 128) {
      scales[kTileM + c] = n0 + c < a.N ? __ldg(a.w_scale + n0 + c) : 0.0f;
      scales[kTileM + BN + c] = a.bias != nullptr && n0 + c < a.N ? __ldg(a.bias + n0 + c) : 0.0f;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");  // the four warps
    const bool ok = wait(done, 0);
    __syncwarp();
    tc_fence_after();
    const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16);
    if (split == 1) {
      // Every load has been consumed: the ring's memory stages the rows.
      if (__all_sync(0xffffffffu, ok)) {
        uint8_t* stage = smem + q * 4096;
        const float xs = scales[row];
        if (a.out_f32)
          drain_rows<true>(taddr, BN, stage, scales + kTileM, scales + kTileM + BN, xs, a, m0 + 32 * q, n0);
        else
          drain_rows<false>(taddr, BN, stage, scales + kTileM, scales + kTileM + BN, xs, a, m0 + 32 * q, n0);
      }
    } else {
      // This CTA's sums, for its cluster (warps whose rows do not exist have none).
      int* stage = reinterpret_cast<int*>(smem) + row * C::PITCH;
#pragma unroll 1
      for (int c0 = m0 + 32 * q < a.M ? 0 : BN; c0 < BN; c0 += 32) {
        uint32_t d[32];
        tmem_ld32(taddr + c0, d);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<int4*>(stage + c0 + j) = make_int4((int)d[j], (int)d[j + 1], (int)d[j + 2], (int)d[j + 3]);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, BN);
  if (split == 1) return;
  cluster_sync();

  // This CTA's share of the tile's rows: the sums of all CTAs of the cluster, scaled.
  const uint32_t there = a.M - m0 < (uint32_t)kTileM ? a.M - m0 : kTileM;
  const int rows = (int)((there + split - 1) / split);
  const int row_lo = (int)rank * rows;
  const bool vec = a.ldo % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % (a.out_f32 ? 16 : 8) == 0;
  // All of a thread's reads are on their way at once, and each CTA begins with its own
  // sums, so that they do not all read the same one's (128 x 4096 x 4096 in pairs: 9.5
  // to 9.0 us).
  auto sum_rows = [&](auto ctas) {
    constexpr uint32_t kSplit = decltype(ctas)::value;
    uint32_t part[kSplit];
#pragma unroll
    for (uint32_t p = 0; p < kSplit; ++p) part[p] = mapa_shared(s_base, (rank + p) % kSplit);
#pragma unroll 2
    for (int i = tid; i < rows * (BN / 4); i += kTileThreads) {
      const int r = row_lo + i / (BN / 4), c = i % (BN / 4) * 4;
      const uint32_t m = m0 + r, n = n0 + c;
      if (r >= (int)there || n >= a.N) continue;
      const uint32_t at = (uint32_t)(r * C::PITCH + c) * 4;
      int4 sums[kSplit];
#pragma unroll
      for (uint32_t p = 0; p < kSplit; ++p) sums[p] = ld_cluster_int4(part[p] + at);
      int4 s = sums[0];
#pragma unroll
      for (uint32_t p = 1; p < kSplit; ++p) {
        s.x += sums[p].x;
        s.y += sums[p].y;
        s.z += sums[p].z;
        s.w += sums[p].w;
      }
      const float xs = scales[r];
      const float4 ws = *reinterpret_cast<const float4*>(scales + kTileM + c);
      float4 v = make_float4(int8_scaled(s.x, xs, ws.x), int8_scaled(s.y, xs, ws.y), int8_scaled(s.z, xs, ws.z),
                             int8_scaled(s.w, xs, ws.w));
      if (a.bias != nullptr) {
        const float4 b = *reinterpret_cast<const float4*>(scales + kTileM + BN + c);
        v = make_float4(int8_biased(v.x, b.x), int8_biased(v.y, b.y), int8_biased(v.z, b.z), int8_biased(v.w, b.w));
      }
      const uint64_t o = (uint64_t)m * a.ldo + n;
      if (a.out_f32) {
        float* out = static_cast<float*>(a.out) + o;
        if (vec && n + 4 <= a.N) {
          *reinterpret_cast<float4*>(out) = v;
        } else {
          out[0] = v.x;
          if (n + 1 < a.N) out[1] = v.y;
          if (n + 2 < a.N) out[2] = v.z;
          if (n + 3 < a.N) out[3] = v.w;
        }
      } else {
        uint16_t* out = static_cast<uint16_t*>(a.out) + o;
        const uint32_t lo = bf16_pair(v.x, v.y), hi = bf16_pair(v.z, v.w);
        if (vec && n + 4 <= a.N) {
          *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
        } else {
          out[0] = (uint16_t)lo;
          if (n + 1 < a.N) out[1] = (uint16_t)(lo >> 16);
          if (n + 2 < a.N) out[2] = (uint16_t)hi;
          if (n + 3 < a.N) out[3] = (uint16_t)(hi >> 16);
        }
      }
    }
  };
  // Tiles of 128 channels are split over four CTAs only.
  if constexpr (BN == 64) {
    if (split == 2) sum_rows(std::integral_constant<uint32_t, 2>());
    if (split == 8) sum_rows(std::integral_constant<uint32_t, 8>());
  }
  if (split == 4) sum_rows(std::integral_constant<uint32_t, 4>());
  // A CTA's sums stay until every CTA of its cluster has read them.
  cluster_sync();
}

namespace {

template <int BN, bool DEEP>
cudaError_t launch_tile(const Int8MatmulArgs& a, uint32_t split, cudaStream_t stream) {
  using C = TileCfg<BN, DEEP>;
  auto kern = int8_tile_kernel<BN, DEEP>;
  cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM);
  if (err != cudaSuccess) return err;
  const uint64_t tiles = (uint64_t)((a.M + kTileM - 1) / kTileM) * ((a.N + BN - 1) / BN);
  if (tiles * split > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  // A batch of fewer than 128 tokens loads only its rows (in eights): the
  // tile's other rows hold whatever was there, and so do their sums, which nobody
  // reads.
  const uint32_t x_rows = a.M < (uint32_t)kTileM ? (a.M + 7) / 8 * 8 : kTileM;
  CUtensorMap x, w;
  err = make_map_2d_pitched(&x, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.M, a.K, a.ldx, x_rows, kStageK,
                            CU_TENSOR_MAP_SWIZZLE_128B);
  if (err != cudaSuccess) return err;
  err = make_map_2d(&w, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.N, a.K, BN, kStageK, CU_TENSOR_MAP_SWIZZLE_128B);
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)(tiles * split));
  if (split == 1) return launch_pdl(kern, grid, dim3(kTileThreads), C::SMEM, stream, a, split, x_rows, x, w);
  return launch_pdl_cluster(kern, grid, dim3(kTileThreads), C::SMEM, split, stream, a, split, x_rows, x, w);
}

}  // namespace

namespace {

constexpr int kPairM = 256, kPairN = 256;
constexpr int kPairThreads = 32 * 10;
constexpr int kPairEpiWarps = 8;

struct PairCfg8 {
  static constexpr int STAGES = 5;
  static constexpr int A_BYTES = kPairM / 2 * kStageK;  // this CTA's token rows
  static constexpr int B_BYTES = kPairN / 2 * kStageK;  // this CTA's half of the channels
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int OFF_ROWS = STAGES * STAGE_BYTES;              // per epilogue warp: staged rows
  static constexpr int OFF_SCALE = OFF_ROWS + kPairEpiWarps * 4096;  // and 128 scales, 128 biases
  static constexpr int OFF_BAR = OFF_SCALE + kPairEpiWarps * 1024;
  // full[STAGES] (first CTA), empty[STAGES], done[2], dfree[2] (first CTA)
  static constexpr int NBAR = 2 * STAGES + 4;
  static constexpr int OFF_TMEM = OFF_BAR + 8 * NBAR;
  static constexpr int OFF_ABORT = OFF_TMEM + 16;
  static constexpr int SMEM = OFF_ABORT + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(2 * (SMEM + 1024) > 228 * 1024, "one CTA per SM: it takes all of its tensor memory");
  static_assert(tc_smem_safe(SMEM, 512), "no pairs of two kernels wait for each other's tensor memory");
};

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    int8_pair_kernel(const Int8MatmulArgs a, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_w) {
  using C = PairCfg8;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t s_base = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (s_base - raw_base);
  const uint32_t full = s_base + C::OFF_BAR;
  const uint32_t empty = full + 8 * C::STAGES;
  const uint32_t done = empty + 8 * C::STAGES;
  const uint32_t dfree = done + 16;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = cluster_ctarank();

  if (tid == 0) {
    tmap_prefetch(&tm_x);
    tmap_prefetch(&tm_w);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int d = 0; d < 2; ++d) {
      mbar_init(done + 8 * d, 1);
      mbar_init(dfree + 8 * d, 2 * kPairEpiWarps);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_holder), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the first CTA's barriers exist before any signal to them
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  const uint32_t tiles_m = (a.M + kPairM - 1) / kPairM, tiles_n = (a.N + kPairN - 1) / kPairN;
  const uint32_t ntile = tiles_m * tiles_n;
  const uint32_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const uint32_t nst = (a.K + kStageK - 1) / kStageK;

  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait(bar, parity)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp == 0) {
    const bool one = elect_one();
    const uint32_t lead_full = mapa_shared(full, 0);
    uint32_t i = 0;
    bool ok = true;
    for (uint32_t t = pair; t < ntile && ok; t += npairs) {
      const int y_x = (int)(t % tiles_m * kPairM + rank * (kPairM / 2));
      const int y_w = (int)(t / tiles_m * kPairN + rank * (kPairN / 2));
      for (uint32_t st = 0; st < nst; ++st, ++i) {
        const uint32_t slot = i % C::STAGES, round = i / C::STAGES;
        ok = round == 0 || __all_sync(0xffffffffu, wait(empty + 8 * slot, (round - 1) & 1));
        if (!ok) break;
        const uint32_t dst = s_base + slot * C::STAGE_BYTES;
        if (one) {
          // The first CTA's barrier counts both CTAs' bytes.
          if (rank == 0) mbar_arrive_expect_tx(full + 8 * slot, 2 * C::STAGE_BYTES);
          tma_load_2d_pair(dst, &tm_x, (int)(st * kStageK), y_x, lead_full + 8 * slot);
          tma_load_2d_pair(dst + C::A_BYTES, &tm_w, (int)(st * kStageK), y_w, lead_full + 8 * slot);
        }
        __syncwarp();
      }
    }
    // The last stages' products read them: wait for those, and in the first CTA
    // for its full barriers, which count both CTAs' bytes.
    for (uint32_t j = i > (uint32_t)C::STAGES ? i - C::STAGES : 0; j < i; ++j) {
      mbar_wait(empty + 8 * (j % C::STAGES), (j / C::STAGES) & 1);
      if (rank == 0) mbar_wait(full + 8 * (j % C::STAGES), (j / C::STAGES) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_s8_s32(kPairM, kPairN);
      const bool one = elect_one();
      uint32_t i = 0, n = 0;
      for (uint32_t t = pair; t < ntile; t += npairs, ++n) {
        const uint32_t db = n & 1;
        if (n >= 2) {
          wait(dfree + 8 * db, (n / 2 - 1) & 1);
          __syncwarp();
          tc_fence_after();
        }
        const uint32_t dcol = tmem + db * kPairN;
        for (uint32_t st = 0; st < nst; ++st, ++i) {
          const uint32_t slot = i % C::STAGES;
          if (!__all_sync(0xffffffffu, wait(full + 8 * slot, (i / C::STAGES) & 1))) break;
          tc_fence_after();
          const uint32_t abase = s_base + slot * C::STAGE_BYTES, bbase = abase + C::A_BYTES;
          if (one) {
#pragma unroll
            for (int k = 0; k < kStageK / 32; ++k)
              tc_mma_pair_s8_ss(dcol, smem_desc_sw128(abase + 32 * k), smem_desc_sw128(bbase + 32 * k), idesc,
                                st > 0 || k > 0 ? 1u : 0u);
            tc_commit_pair(empty + 8 * slot, 0x3);
          }
          __syncwarp();
        }
        if (one) tc_commit_pair(done + 8 * db, 0x3);
        __syncwarp();
      }
      // No product may still run when the tensor memory is freed.
      if (n > 0) mbar_wait(done + 8 * ((n - 1) & 1), ((n - 1) / 2) & 1);
      __syncwarp();
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;
    const uint32_t lead_dfree = mapa_shared(dfree, 0);
    float* scale = reinterpret_cast<float*>(smem + C::OFF_SCALE) + (warp - 2) * 256;
    uint8_t* stage = smem + C::OFF_ROWS + (warp - 2) * 4096;
    uint32_t n = 0;
    for (uint32_t t = pair; t < ntile; t += npairs, ++n) {
      const uint32_t db = n & 1;
      const uint32_t m0 = t % tiles_m * kPairM + rank * (kPairM / 2) + 32 * q;
      const uint32_t n0 = t / tiles_m * kPairN + half * (kPairN / 2);
      // This tile's scales, while its products run.
      const float xs = m0 + lane < a.M ? __ldg(a.x_scale + m0 + lane) : 0.0f;
#pragma unroll
      for (int c = lane; c < kPairN / 2; c += 32) {
        scale[c] = n0 + c < a.N ? __ldg(a.w_scale + n0 + c) : 0.0f;
        scale[128 + c] = a.bias != nullptr && n0 + c < a.N ? __ldg(a.bias + n0 + c) : 0.0f;
      }
      __syncwarp();
      bool ok = wait(done + 8 * db, (n / 2) & 1);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const uint32_t dcol = tmem + lane_off + db * kPairN + half * (kPairN / 2);
      if (ok) {
        if (a.out_f32) drain_rows<true>(dcol, kPairN / 2, stage, scale, scale + 128, xs, a, m0, n0);
        else drain_rows<false>(dcol, kPairN / 2, stage, scale, scale + 128, xs, a, m0, n0);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(lead_dfree + 8 * db);
    }
  }

  __syncthreads();
  __syncwarp();
  cluster_sync();  // no more remote arrives, and the pair's products are done
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, 512);
  }
}

cudaError_t launch_int8_pair(const Int8MatmulArgs& a, cudaStream_t stream) {
  using C = PairCfg8;
  cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(int8_pair_kernel), C::SMEM);
  if (err != cudaSuccess) return err;
  const uint64_t tiles = (uint64_t)((a.M + kPairM - 1) / kPairM) * ((a.N + kPairN - 1) / kPairN);
  if (tiles > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  uint64_t pairs = (uint64_t)sm_count() / 2;
  if (pairs > tiles) pairs = tiles;
  CUtensorMap x, w;
  err = make_map_2d_pitched(&x, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.M, a.K, a.ldx, kPairM / 2, kStageK,
                            CU_TENSOR_MAP_SWIZZLE_128B);
  if (err != cudaSuccess) return err;
  err = make_map_2d(&w, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.N, a.K, kPairN / 2, kStageK,
                    CU_TENSOR_MAP_SWIZZLE_128B);
  if (err != cudaSuccess) return err;
  return launch_pdl(int8_pair_kernel, dim3((unsigned)(2 * pairs)), dim3(kPairThreads), C::SMEM, stream, a, x, w);
}

int int8_tile_slots(uint32_t split) {
  const int sms = sm_count();
  if (split < 4) return sms;
  // The answer for a device does not change: asked once.
  static std::atomic<int> known[64][2];
  int dev = 0, clusters = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sms * 3 / 4;
  std::atomic<int>& slots = known[dev][split == 8];
  if (const int n = slots.load(std::memory_order_relaxed)) return n;
  using C = TileCfg<64, true>;
  const void* kern = reinterpret_cast<const void*>(int8_tile_kernel<64, true>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (ensure_dynamic_smem(kern, C::SMEM) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess || clusters < 1) {
    cudaGetLastError();
    clusters = sms * 3 / 4 / (int)split;
  }
  slots.store(clusters * (int)split, std::memory_order_relaxed);
  return clusters * (int)split;
}

bool int8_tile_deep(uint32_t M, uint32_t N, uint32_t bn, uint32_t split) {
  const uint64_t ctas = (uint64_t)((M + kTileM - 1) / kTileM) * ((N + bn - 1) / bn) * split;
  return ctas <= (uint64_t)int8_tile_slots(split);
}

cudaError_t launch_int8_tile(const Int8MatmulArgs& a, const Int8Form& f, cudaStream_t stream) {
  if (f.channels == 64)
    return f.deep ? launch_tile<64, true>(a, f.split, stream) : launch_tile<64, false>(a, f.split, stream);
  return f.deep ? launch_tile<128, true>(a, f.split, stream) : launch_tile<128, false>(a, f.split, stream);
}

cudaError_t read_int8_error(int* value, bool clear) { return read_error_word(&g_device_error, value, clear); }

}  // namespace nvm
