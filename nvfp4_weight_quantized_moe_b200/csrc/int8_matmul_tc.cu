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
// Every wait is bounded; on timeout a CTA flags the device error word and skips
// its remaining waits.

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace nvm {

namespace {

constexpr int kStageK = 128;   // bytes of K per stage: one swizzled row
constexpr int kTileM = 128;

NVM_DEV float scaled(int sum, float xs, float ws) { return (float)sum * xs * ws; }

NVM_DEV uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

NVM_DEV void store_one(void* out, bool f32, uint64_t at, float v) {
  if (f32) {
    static_cast<float*>(out)[at] = v;
  } else {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    static_cast<uint16_t*>(out)[at] = *reinterpret_cast<const uint16_t*>(&b);
  }
}
// Four consecutive outputs at an address that is a multiple of their size.
NVM_DEV void store_four(void* out, bool f32, uint64_t at, const float (&v)[4]) {
  if (f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
        make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
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
NVM_DEV int ld_cluster_int(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int BN>
struct TileCfg {
  static constexpr int STAGES = BN == 128 ? 3 : 4;
  static constexpr int A_BYTES = kTileM * kStageK;
  static constexpr int B_BYTES = BN * kStageK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int PITCH = BN + 4;  // ints between rows of the staged sums
  static constexpr int OFF_BAR = STAGES * STAGE_BYTES;
  // full[STAGES], empty[STAGES], done
  static constexpr int NBAR = 2 * STAGES + 1;
  static constexpr int OFF_TMEM = OFF_BAR + 8 * NBAR;
  static constexpr int OFF_ABORT = OFF_TMEM + 16;
  static constexpr int SMEM = OFF_ABORT + 16 + 1024;
  static_assert(kTileM * PITCH * 4 <= OFF_BAR, "staged sums fit the ring");
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
  // Two CTAs of this size are all an SM holds, with anything that shares it: no
  // allocation of tensor memory ever waits for another cluster's.
  static_assert(3 * (SMEM + 1024) > 228 * 1024 && 2 * BN <= 512, "tensor memory");
};

constexpr int kTileThreads = 192;  // warp 0 loads, warp 1 issues, warps 2-5 drain

}  // namespace

template <int BN>
__global__ void __launch_bounds__(kTileThreads)
    int8_tile_kernel(const Int8MatmulArgs a, const uint32_t split, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_w) {
  using C = TileCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t s_base = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (s_base - raw_base);
  const uint32_t full = s_base + C::OFF_BAR;
  const uint32_t empty = full + 8 * C::STAGES;
  const uint32_t done = empty + 8 * C::STAGES;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
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
    if (lane == 0) {
      uint32_t i = 0;
      for (uint32_t st = st_lo; st < st_hi; ++st, ++i) {
        const uint32_t slot = i % C::STAGES, round = i / C::STAGES;
        if (round > 0 && !wait(empty + 8 * slot, (round - 1) & 1)) break;
        const uint32_t dst = s_base + slot * C::STAGE_BYTES, bar = full + 8 * slot;
        mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
        tma_load_2d(dst, &tm_x, (int)(st * kStageK), (int)m0, bar);
        tma_load_2d(dst + C::A_BYTES, &tm_w, (int)(st * kStageK), (int)n0, bar);
      }
      // Nothing may still land in this CTA's memory when it goes on.
      for (uint32_t j = i > (uint32_t)C::STAGES ? i - C::STAGES : 0; j < i; ++j)
        mbar_wait(full + 8 * (j % C::STAGES), (j / C::STAGES) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_s8_s32(kTileM, BN);
      uint32_t i = 0;
      for (uint32_t st = st_lo; st < st_hi; ++st, ++i) {
        const uint32_t slot = i % C::STAGES;
        if (!wait(full + 8 * slot, (i / C::STAGES) & 1)) break;
        tc_fence_after();
        const uint32_t abase = s_base + slot * C::STAGE_BYTES, bbase = abase + C::A_BYTES;
#pragma unroll
        for (int k = 0; k < kStageK / 32; ++k)
          tc_mma_s8_ss(tmem, smem_desc_sw128(abase + 32 * k), smem_desc_sw128(bbase + 32 * k), idesc,
                       i > 0 || k > 0 ? 1u : 0u);
        tc_commit(empty + 8 * slot);
      }
      tc_commit(done);
      mbar_wait(done, 0);  // no MMA may still run when the tensor memory is freed
    }
    __syncwarp();
  } else {
    wait(done, 0);
    __syncwarp();
    tc_fence_after();
    // This CTA's sums into the ring's memory (every load has been consumed).
    const int q = warp & 3, row = 32 * q + lane;
    int* stage = reinterpret_cast<int*>(smem) + row * C::PITCH;
#pragma unroll 1
    for (int c0 = 0; c0 < BN; c0 += 32) {
      uint32_t d[32];
      tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + c0, d);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<int4*>(stage + c0 + j) = make_int4((int)d[j], (int)d[j + 1], (int)d[j + 2], (int)d[j + 3]);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (split > 1) cluster_sync();
  if (warp == 1) tmem_dealloc(tmem, BN);

  // Rows row_lo .. of the tile: the sums of all CTAs of the cluster, scaled.
  const int rows = kTileM / (int)split;
  const int row_lo = (int)rank * rows;
  const bool vec = a.ldo % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % (a.out_f32 ? 16 : 8) == 0;
  if (vec) {
    for (int i = tid; i < rows * (BN / 4); i += kTileThreads) {
      const int r = row_lo + i / (BN / 4), c = i % (BN / 4) * 4;
      const uint32_t m = m0 + r, n = n0 + c;
      if (m >= a.M || n >= a.N) continue;
      const uint32_t at = s_base + (uint32_t)(r * C::PITCH + c) * 4;
      int4 s = make_int4(0, 0, 0, 0);
      if (split == 1) {
        s = *reinterpret_cast<const int4*>(smem + (at - s_base));
      } else {
        for (uint32_t p = 0; p < split; ++p) {
          const int4 v = ld_cluster_int4(mapa_shared(at, p));
          s.x += v.x;
          s.y += v.y;
          s.z += v.z;
          s.w += v.w;
        }
      }
      const float xs = __ldg(a.x_scale + m);
      const int sums[4] = {s.x, s.y, s.z, s.w};
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = 0.0f;
        if (n + j < a.N) {
          v[j] = scaled(sums[j], xs, __ldg(a.w_scale + n + j));
          if (a.bias != nullptr) v[j] += __ldg(a.bias + n + j);
        }
      }
      const uint64_t o = (uint64_t)m * a.ldo + n;
      if (n + 4 <= a.N) {
        store_four(a.out, a.out_f32, o, v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < a.N) store_one(a.out, a.out_f32, o + j, v[j]);
      }
    }
  } else {
    for (int i = tid; i < rows * BN; i += kTileThreads) {
      const int r = row_lo + i / BN, c = i % BN;
      const uint32_t m = m0 + r, n = n0 + c;
      if (m >= a.M || n >= a.N) continue;
      const uint32_t at = s_base + (uint32_t)(r * C::PITCH + c) * 4;
      int s = 0;
      if (split == 1) {
        s = *reinterpret_cast<const int*>(smem + (at - s_base));
      } else {
        for (uint32_t p = 0; p < split; ++p) s += ld_cluster_int(mapa_shared(at, p));
      }
      float v = scaled(s, __ldg(a.x_scale + m), __ldg(a.w_scale + n));
      if (a.bias != nullptr) v += __ldg(a.bias + n);
      store_one(a.out, a.out_f32, (uint64_t)m * a.ldo + n, v);
    }
  }
  // A CTA's sums stay until every CTA of its cluster has read them.
  if (split > 1) cluster_sync();
}

namespace {

template <int BN>
cudaError_t launch_tile(const Int8MatmulArgs& a, uint32_t split, cudaStream_t stream) {
  using C = TileCfg<BN>;
  auto kern = int8_tile_kernel<BN>;
  cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM);
  if (err != cudaSuccess) return err;
  const uint64_t tiles = (uint64_t)((a.M + kTileM - 1) / kTileM) * ((a.N + BN - 1) / BN);
  if (tiles * split > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  CUtensorMap x, w;
  err = make_map_2d_pitched(&x, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.M, a.K, a.ldx, kTileM, kStageK,
                            CU_TENSOR_MAP_SWIZZLE_128B);
  if (err != cudaSuccess) return err;
  err = make_map_2d(&w, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.N, a.K, BN, kStageK, CU_TENSOR_MAP_SWIZZLE_128B);
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)(tiles * split));
  if (split == 1) return launch_pdl(kern, grid, dim3(kTileThreads), C::SMEM, stream, a, split, x, w);
  return launch_pdl_cluster(kern, grid, dim3(kTileThreads), C::SMEM, split, stream, a, split, x, w);
}

}  // namespace

namespace {

constexpr int kPairM = 256, kPairN = 256;
constexpr int kPairThreads = 32 * 10;
constexpr int kPairEpiWarps = 8;

struct PairCfg8 {
  static constexpr int STAGES = 6;
  static constexpr int A_BYTES = kPairM / 2 * kStageK;  // this CTA's token rows
  static constexpr int B_BYTES = kPairN / 2 * kStageK;  // this CTA's half of the channels
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int OFF_SCALE = STAGES * STAGE_BYTES;  // per epilogue warp: 32 scales, 32 biases
  static constexpr int OFF_BAR = OFF_SCALE + kPairEpiWarps * 256;
  // full[STAGES] (first CTA), empty[STAGES], done[2], dfree[2] (first CTA)
  static constexpr int NBAR = 2 * STAGES + 4;
  static constexpr int OFF_TMEM = OFF_BAR + 8 * NBAR;
  static constexpr int OFF_ABORT = OFF_TMEM + 16;
  static constexpr int SMEM = OFF_ABORT + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(2 * (SMEM + 1024) > 228 * 1024, "one CTA per SM: it takes all of its tensor memory");
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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();

  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) {
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
    if (lane == 0) {
      const uint32_t lead_full = mapa_shared(full, 0);
      uint32_t i = 0;
      for (uint32_t t = pair; t < ntile && !*abort_flag; t += npairs) {
        const int y_x = (int)(t % tiles_m * kPairM + rank * (kPairM / 2));
        const int y_w = (int)(t / tiles_m * kPairN + rank * (kPairN / 2));
        for (uint32_t st = 0; st < nst; ++st, ++i) {
          const uint32_t slot = i % C::STAGES, round = i / C::STAGES;
          if (round > 0 && !wait(empty + 8 * slot, (round - 1) & 1)) break;
          const uint32_t dst = s_base + slot * C::STAGE_BYTES;
          // The first CTA's barrier counts both CTAs' bytes.
          if (rank == 0) mbar_arrive_expect_tx(full + 8 * slot, 2 * C::STAGE_BYTES);
          tma_load_2d_pair(dst, &tm_x, (int)(st * kStageK), y_x, lead_full + 8 * slot);
          tma_load_2d_pair(dst + C::A_BYTES, &tm_w, (int)(st * kStageK), y_w, lead_full + 8 * slot);
        }
      }
      // The last stages' products read them: wait for those, and in the first CTA
      // for its full barriers, which count both CTAs' bytes.
      for (uint32_t j = i > (uint32_t)C::STAGES ? i - C::STAGES : 0; j < i; ++j) {
        mbar_wait(empty + 8 * (j % C::STAGES), (j / C::STAGES) & 1);
        if (rank == 0) mbar_wait(full + 8 * (j % C::STAGES), (j / C::STAGES) & 1);
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc = idesc_s8_s32(kPairM, kPairN);
      uint32_t i = 0, n = 0;
      for (uint32_t t = pair; t < ntile; t += npairs, ++n) {
        const uint32_t db = n & 1;
        if (n >= 2) {
          wait(dfree + 8 * db, (n / 2 - 1) & 1);
          tc_fence_after();
        }
        const uint32_t dcol = tmem + db * kPairN;
        for (uint32_t st = 0; st < nst; ++st, ++i) {
          const uint32_t slot = i % C::STAGES;
          if (!wait(full + 8 * slot, (i / C::STAGES) & 1)) break;
          tc_fence_after();
          const uint32_t abase = s_base + slot * C::STAGE_BYTES, bbase = abase + C::A_BYTES;
#pragma unroll
          for (int k = 0; k < kStageK / 32; ++k)
            tc_mma_pair_s8_ss(dcol, smem_desc_sw128(abase + 32 * k), smem_desc_sw128(bbase + 32 * k), idesc,
                              st > 0 || k > 0 ? 1u : 0u);
          tc_commit_pair(empty + 8 * slot, 0x3);
        }
        tc_commit_pair(done + 8 * db, 0x3);
      }
      // No product may still run when the tensor memory is freed.
      if (n > 0) mbar_wait(done + 8 * ((n - 1) & 1), ((n - 1) / 2) & 1);
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;
    const uint32_t lead_dfree = mapa_shared(dfree, 0);
    float* scale = reinterpret_cast<float*>(smem + C::OFF_SCALE) + (warp - 2) * 64;
    const uint64_t elem = a.out_f32 ? 4 : 2;
    const bool vec = a.ldo * elem % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
    uint32_t n = 0;
    for (uint32_t t = pair; t < ntile; t += npairs, ++n) {
      const uint32_t db = n & 1;
      const uint32_t m = t % tiles_m * kPairM + rank * (kPairM / 2) + 32 * q + lane;
      const uint32_t n_lo = t / tiles_m * kPairN + half * (kPairN / 2);
      const float xs = m < a.M ? __ldg(a.x_scale + m) : 0.0f;
      bool ok = wait(done + 8 * db, (n / 2) & 1);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const uint32_t dcol = tmem + lane_off + db * kPairN + half * (kPairN / 2);
#pragma unroll 1
      for (int c0 = 0; c0 < kPairN / 2; c0 += 32) {
        const uint32_t n0 = n_lo + c0;
        if (n0 >= a.N) break;
        __syncwarp();
        scale[lane] = n0 + lane < a.N ? __ldg(a.w_scale + n0 + lane) : 0.0f;
        scale[32 + lane] = a.bias != nullptr && n0 + lane < a.N ? __ldg(a.bias + n0 + lane) : 0.0f;
        __syncwarp();
        uint32_t d[32];
        tmem_ld32(dcol + c0, d);
        tmem_wait_ld();
        if (!ok || m >= a.M) continue;
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = scaled((int)d[j], xs, scale[j]);
        if (a.bias != nullptr) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += scale[32 + j];
        }
        const uint64_t o = (uint64_t)m * a.ldo + n0;
        if (vec && n0 + 32 <= a.N) {
          if (a.out_f32) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.out) + o);
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          } else {
            uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + o);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              p[j] = make_uint4(bf16_pair(v[8 * j], v[8 * j + 1]), bf16_pair(v[8 * j + 2], v[8 * j + 3]),
                                bf16_pair(v[8 * j + 4], v[8 * j + 5]), bf16_pair(v[8 * j + 6], v[8 * j + 7]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (n0 + j < a.N) store_one(a.out, a.out_f32, o + j, v[j]);
        }
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

cudaError_t launch_int8_tile(const Int8MatmulArgs& a, int bn, uint32_t split, cudaStream_t stream) {
  return bn == 64 ? launch_tile<64>(a, split, stream) : launch_tile<128>(a, split, stream);
}

cudaError_t read_int8_error(int* value, bool clear) { return read_error_word(&g_device_error, value, clear); }

}  // namespace nvm
