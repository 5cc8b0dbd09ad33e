// Matrix products with an epilogue: y = act(x W^T + bias) + residual, bf16 in and out, fp32 sums.
//
// x [T, K] and W [M, K] are K-major, so both operands come from memory in the tensor cores' own order (128-byte swizzled
// slabs of 64 elements of K, by TMA; what lies past an extent arrives as zeros). Bias, activation and residual are applied
// to the fp32 sum and the result is rounded to bf16 once.
//
// gemm_pair_kernel: many rows. Two SMs work as one tensor-core pair (tcgen05 .cta_group::2) on a tile of 256 rows x 256
// columns (or fewer, a multiple of 32): each holds its 128 rows of x and half of W's 256 rows of a slab, 32 KB a step of
// 64 in K for 2 x 256 x 256 x 64 operations, half of what two single SMs would move. Sums lie in TMEM twice, so that one
// tile's epilogue runs under the next one's products. Bound by the tensor cores: 4096 x 16384 x 8192 in 573 us
// for a few calls (1.92 PFLOP/s), in a loop 600 to 690 by what the power limit leaves (cuBLAS likewise: 568, and in turn in a loop
// 642 to 669 beside 651 to 657); 4096 x 4096 x 4096 in 79 us. Six stages of one slab (three of two:
// 83.6 us against 80.1 of the last; five: 82.2); one staging slab a warp makes room for the sixth.
//
// gemm_narrow_kernel: few rows. Bound by W's bytes, so W takes the M side of the instruction (128 of its rows a CTA) and
// the rows of x the N side (16 to 128), and K is split over the CTAs of a cluster, whose sums meet through distributed
// shared memory in the order of their ranks: no workspace, no atomics, the same result every time. 1 x 16384 x 8192 in
// 42.4 us (6.3 TB/s, 93 % of a copy's), 64 rows 45; what the wider x costs is mostly the exchange of sums.
#include <cstdint>
#include <cuda_runtime.h>

#include "decode_common.cuh"
#include "mla_kernels.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

// What the epilogue does: bias and residual; an activation between them; or keys and values of the heads.
enum { kPlain = 0, kSilu = 1, kGelu = 2, kKeysValues = 3 };
// of values (kKeysValues): their scale, and the bits of the magnitudes that fp16 takes
constexpr float kValueScale = 1 << kValueLog2;
constexpr uint32_t kValueMin = (127u + kValueMinLog2) << 23, kValueMax = (127u + kValueMaxLog2) << 23;

__device__ __forceinline__ float2 mul2(float2 a, float b) { return fma2(a, b, make_float2(0.f, 0.f)); }
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The activation of two sums, in packed instructions where there are any.
template <int KIND>
__device__ __forceinline__ float2 activate(float2 y) {
  constexpr float kLog2e = 1.4426950408889634f;
  if (KIND == kSilu) {
    const float2 e = mul2(y, -kLog2e);
    return make_float2(y.x * fast_rcp(1.f + fast_exp2(e.x)), y.y * fast_rcp(1.f + fast_exp2(e.y)));
  }
  if (KIND != kGelu) return y;
  // y Phi(y) = y erfc(-y / sqrt 2) / 2, from the side where nothing cancels: with z = |y| / sqrt 2, erfc(z) = t e^(P(t) - z^2),
  // t = 1 / (1 + z / 2), fractional error below 1.2e-7: the Chebyshev fit of Press, Teukolsky, Vetterling and Flannery,
  // Numerical Recipes in C, 2nd ed., section 6.2 (erfcc)
  const float2 z = mul2(make_float2(fabsf(y.x), fabsf(y.y)), 0.70710678118654752f);
  const float2 d = fma2(z, 0.5f, make_float2(1.f, 1.f));
  const float2 t = make_float2(fast_rcp(d.x), fast_rcp(d.y));
  constexpr float kP[9] = {-0.82215223f, 1.48851587f, -1.13520398f, 0.27886807f, -0.18628806f,
                           0.09678418f, 0.37409196f, 1.00002368f, -1.26551223f};
  float2 p = make_float2(0.17087277f, 0.17087277f);
#pragma unroll
  for (int i = 0; i < 9; ++i) p = fma2v(t, p, make_float2(kP[i], kP[i]));
  p = mul2(fma2v(make_float2(-z.x, -z.y), z, p), kLog2e);
  const float2 half = make_float2(0.5f * t.x * fast_exp2(p.x), 0.5f * t.y * fast_exp2(p.y));
  return make_float2(y.x * (y.x < 0.f ? half.x : 1.f - half.x), y.y * (y.y < 0.f ? half.y : 1.f - half.y));
}

// ----------------------------------------------------------------------------- CTA pairs
constexpr int kGemmThreads = 320;              // TMA, MMA, 8 epilogue warps
constexpr int kGemmStages = 6;
constexpr uint32_t kGemmA = 128 * 128;         // this CTA's 128 rows of x, 64 of K
constexpr uint32_t kGemmB = 128 * 128;         // its half of W's 256 rows
constexpr uint32_t kGemmStage = kGemmA + kGemmB;
constexpr uint32_t kGemmOffStaging = kGemmStages * kGemmStage;
constexpr uint32_t kGemmSlab = 32 * 128;       // 32 rows x 64 columns of the result: one warp's store
constexpr uint32_t kGemmOffMisc = kGemmOffStaging + 8 * kGemmSlab;

struct GemmMisc {
  uint64_t full[kGemmStages], empty[kGemmStages];  // full: in the even CTA, both CTAs' bytes
  uint64_t acc_full[2], acc_empty[2];              // acc_empty: in the even CTA, 16 warps
  uint64_t last;
  uint32_t tmem_base;
  int abort;
  unsigned int status;  // where the caller gave none
};
constexpr size_t kGemmSmem = kGemmOffMisc + sizeof(GemmMisc) + 1024;
static_assert(kGemmSmem <= 232448, "shared memory budget of one CTA");

// 32 rows x 64 columns, a row a lane, leave through the warp's slab of shared memory by TMA, as whole 128-byte lines: the slab
// is free, 16-byte chunk q (of 8) of a lane's row goes to it, all of it leaves.
__device__ __forceinline__ void slab_free(int lane) {
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
}
__device__ __forceinline__ void slab_put(uint32_t slab, int lane, int q, const uint32_t* o) {
  st_shared_v4(slab + lane * 128 + ((q ^ (lane & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
}
__device__ __forceinline__ void slab_leave(const CUtensorMap* map, uint32_t slab, int lane, int col0, int row0) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, slab, col0, row0);
    bulk_commit();
  }
}

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    gemm_pair_kernel(const __grid_constant__ GemmParams P, const __grid_constant__ CUtensorMap x_map,
                     const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap y_map) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  GemmMisc* misc = reinterpret_cast<GemmMisc*>(smem + kGemmOffMisc);
  volatile int* abort_flag = &misc->abort;
  unsigned int* status = P.status != nullptr ? P.status : &misc->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  auto lead = [&](uint64_t* b) -> uint32_t { return map_shared_rank(smem_addr(b), 0); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGemmStages; ++s) {
      mbar_init(smem_addr(&misc->full[s]), 2);
      mbar_init(smem_addr(&misc->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&misc->acc_full[b]), 1);
      mbar_init(smem_addr(&misc->acc_empty[b]), 16);
    }
    mbar_init(smem_addr(&misc->last), 1);
    misc->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&x_map);
    tma_prefetch_desc(&w_map);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(&misc->tmem_base), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any remote arrive
  tc_fence_after();
  pdl_trigger();
  pdl_wait();
  const uint32_t tmem = misc->tmem_base;
  const int tiles = P.m_tiles * P.n_tiles;
  const int step = static_cast<int>(num_clusters_x());
  // Tiles in bands of `band` row tiles, row tiles fastest: the pairs that run at once share both operands through L2.
  auto place = [&](int t, int* m0, int* n0) {
    const int b = t / (P.band * P.n_tiles), r = t - b * P.band * P.n_tiles;
    const int h = min(P.band, P.m_tiles - b * P.band);
    *m0 = (b * P.band + r % h) * 256;
    *n0 = (r / h) * P.tile_cols;
  };

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = cluster_id_x(); t < tiles && ok; t += step) {
        int m0, n0;
        place(t, &m0, &n0);
        for (int k = 0; k < P.k_blocks; ++k, ++it) {
          const int s = it % kGemmStages;
          const uint32_t a = sb + s * kGemmStage;
          if (it >= kGemmStages &&
              !wait_bar(smem_addr(&misc->empty[s]), (it / kGemmStages - 1) & 1, abort_flag, status)) {
            ok = false;
            break;
          }
          const uint32_t full = lead(&misc->full[s]);
          mbar_arrive_expect_tx_cluster(full, kGemmA + P.tile_cols * 64);
          tma_load_2d_pair(a, &x_map, 64 * k, m0 + 128 * rank, full);
          tma_load_2d_pair(a + kGemmA, &w_map, 64 * k, P.w_row0 + n0 + (P.tile_cols >> 1) * rank, full);
        }
      }
      if (*abort_flag && rank == 0)  // copies still in flight land on this CTA's barriers: wait for them (bounded)
        for (int k = 1; k <= kGemmStages && it - k >= 0; ++k)
          mbar_wait_drain_cluster(smem_addr(&misc->full[(it - k) % kGemmStages]), ((it - k) / kGemmStages) & 1);
    }
  } else if (warp == 1) {
    // (the whole warp goes through the loop, so that descriptors stay in uniform registers)
    if (rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(256, P.tile_cols, 0, 0);
      const uint64_t kmaj = sdesc_sw128(0, 16, 1024);
      int s = 0, u = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = cluster_id_x(); t < tiles && ok; t += step, ++u) {
        const int buf = u & 1;
        if (u >= 2 && !wait_bar(smem_addr(&misc->acc_empty[buf]), ((u >> 1) - 1) & 1, abort_flag, status)) break;
        tc_fence_after();
        for (int k = 0; k < P.k_blocks; ++k) {
          if (!wait_bar(smem_addr(&misc->full[s]), phase, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t a = kmaj | ((sb + s * kGemmStage) >> 4);
            const uint64_t b = kmaj | ((sb + s * kGemmStage + kGemmA) >> 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_bf16_pair(tmem + buf * 256, a + 2 * i, b + 2 * i, idesc, (k | i) ? 1u : 0u);
            mma_commit_pair(smem_addr(&misc->empty[s]), 3);
          }
          __syncwarp();
          if (++s == kGemmStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (ok && elect_one()) mma_commit_pair(smem_addr(&misc->acc_full[buf]), 3);
        __syncwarp();
      }
      if (elect_one()) {
        mma_commit_pair(smem_addr(&misc->last), 1);
        mbar_wait_drain_cluster(smem_addr(&misc->last), 0);
      }
      __syncwarp();
    }
  } else {
    // Epilogue: a warp reaches the TMEM lanes 32 (warp % 4) .. + 31, one row a lane, and takes half
    // of the tile's columns (in products, every other 64).
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t staging = sb + kGemmOffStaging + (warp - 2) * kGemmSlab;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    int u = 0;
    uint4 ahead[8];  // (but for gelu) the residual of the columns that come next
    auto load_residual = [&](int m0, int col0, int width) {
      const int row = m0 + 128 * rank + 32 * quarter + lane;
      const int chunks = P.residual != nullptr && row < P.rows ? min(width, P.cols - col0) >> 3 : 0;
      const uint16_t* rp = P.residual + row * P.residual_stride + col0;
#pragma unroll
      for (int q = 0; q < 8; ++q) ahead[q] = q < chunks ? *reinterpret_cast<const uint4*>(rp + 8 * q) : make_uint4(0, 0, 0, 0);
    };
    for (int t = cluster_id_x(); t < tiles; t += step, ++u) {
      int m0, n0;
      place(t, &m0, &n0);
      if (KIND != kKeysValues && KIND != kGelu && u == 0) load_residual(m0, n0 + 64 * half, 64);
      const int buf = u & 1;
      const int row0 = m0 + 128 * rank + 32 * quarter;
      const uint32_t src = tmem + buf * 256 + lane_off;
      if (!wait_bar(smem_addr(&misc->acc_full[buf]), (u >> 1) & 1, abort_flag, status)) break;
      tc_fence_after();
      if (KIND == kKeysValues) {
        // a tile is one head: 128 columns of its keys, 128 of its values. 32 rows of values leave as fp16 (three bits more than
        // bf16) where their largest is of a size that fp16 holds well, else as bf16, which takes any.
        if (row0 < P.rows) {
          uint32_t acc[128], o[32];
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld32(src + 128 * half + 32 * k, acc + 32 * k);
          tmem_wait_ld();
          bool wide = true;  // (keys are bf16)
          if (half == 1) {
            float largest = 0.f;
#pragma unroll
            for (int k = 0; k < 128; k += 2) {
              const float a = __uint_as_float(acc[k]), b = __uint_as_float(acc[k + 1]);
              largest = max3(largest, fabsf(a), fabsf(b));
              acc[k] = __float_as_uint(a * kValueScale);
              acc[k + 1] = __float_as_uint(b * kValueScale);
            }
            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(largest));  // (as integers)
            wide = top != 0u && (top < kValueMin || top >= kValueMax);
            if (lane == 0) {
              P.value_wide[static_cast<int64_t>(n0 >> 8) * P.value_wide_stride + (row0 >> 5)] = wide;
              if (wide) *P.any_wide = 1;
            }
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float a = __uint_as_float(acc[64 * c + 2 * k]), b = __uint_as_float(acc[64 * c + 2 * k + 1]);
              o[k] = wide ? f32x2_to_bf16x2(a, b) : f32x2_to_f16x2(a, b);
            }
            slab_free(lane);
#pragma unroll
            for (int q = 0; q < 8; ++q) slab_put(staging, lane, q, o + 4 * q);
            slab_leave(&y_map, staging, lane, n0 + 128 * half + 64 * c, row0);
          }
        }
      } else {
#pragma unroll 1
        for (int c = half; 64 * c < P.tile_cols; c += 2) {
          const int col0 = n0 + 64 * c;
          if (row0 >= P.rows || col0 >= P.cols) break;  // (the same in all lanes)
          const int row = row0 + lane;
          const int width = min(64, P.tile_cols - 64 * c);           // 64, or 32 in the last of them
          const int chunks = min(width, P.cols - col0) >> 3;         // of 8 columns
          const bool add = P.residual != nullptr && row < P.rows;
          const uint16_t* rp = P.residual + row * P.residual_stride + col0;
          if (width == 64) slab_free(lane);
          // kPart columns at a time: all of them where little is done to them; 16 with gelu, of which 64 make long code (1001 x 1544 x
          // 6152: 27.5 us against 26.5; silu 24.3 against 25.6)
          constexpr int kPart = KIND == kGelu ? 16 : 64;
#pragma unroll 1
          for (int part = 0; part < 64 / kPart; ++part) {
            uint32_t acc[kPart], o[kPart / 2];
            uint4 res[kPart / 8];
            const int q0 = part * (kPart / 8);  // first 16-byte chunk
            if (kPart == 64) {
              tmem_ld32(src + 64 * c, acc);
              tmem_ld32(src + 64 * c + 32, acc + kPart / 2);
            } else {
              tmem_ld16(src + 64 * c + kPart * part, reinterpret_cast<uint32_t(&)[16]>(acc));
            }
#pragma unroll
            for (int q = 0; q < kPart / 8; ++q) {
              if (KIND != kGelu) res[q] = ahead[q];
              else res[q] = add && q0 + q < chunks ? *reinterpret_cast<const uint4*>(rp + 8 * (q0 + q)) : make_uint4(0, 0, 0, 0);
            }
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < kPart / 8; ++q) {
              const uint4 bu = P.bias != nullptr && q0 + q < chunks ? *reinterpret_cast<const uint4*>(P.bias + col0 + 8 * (q0 + q))
                                                                    : make_uint4(0, 0, 0, 0);
              const uint32_t bh[4] = {bu.x, bu.y, bu.z, bu.w}, rh[4] = {res[q].x, res[q].y, res[q].z, res[q].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float2 y = make_float2(__uint_as_float(acc[8 * q + 2 * i]), __uint_as_float(acc[8 * q + 2 * i + 1]));
                if (P.bias != nullptr)
                  y = add2(y, make_float2(__uint_as_float(bh[i] << 16), __uint_as_float(bh[i] & 0xFFFF0000u)));
                y = activate<KIND>(y);
                if (P.residual != nullptr)
                  y = add2(y, make_float2(__uint_as_float(rh[i] << 16), __uint_as_float(rh[i] & 0xFFFF0000u)));
                o[4 * q + i] = f32x2_to_bf16x2(y.x, y.y);
              }
            }
            // the residual of the next columns while these leave
            if (KIND != kGelu && 64 * (c + 2) < P.tile_cols)
              load_residual(m0, n0 + 64 * (c + 2), min(64, P.tile_cols - 64 * (c + 2)));
#pragma unroll
            for (int q = 0; q < kPart / 8; ++q) {
              if (width == 64) slab_put(staging, lane, q0 + q, o + 4 * q);
              else if (q0 + q < chunks && row < P.rows)
                reinterpret_cast<uint4*>(P.out + row * P.out_stride + col0)[q0 + q] =
                    make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
          }
          if (width == 64) slab_leave(&y_map, staging, lane, col0, row0);
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(lead(&misc->acc_empty[buf]));
      if (KIND != kKeysValues && KIND != kGelu && t + step < tiles) {
        place(t + step, &m0, &n0);
        load_residual(m0, n0 + 64 * half, 64);
      }
    }
    if (lane == 0) bulk_wait<0>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the even CTA's MMAs into both CTAs' TMEM have completed
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ----------------------------------------------------------------------------- few rows
constexpr int kNarrowThreads = 192;

struct NarrowMisc {
  uint64_t full[16], empty[16], acc_full;
  uint32_t tmem_base;
  int abort;
  unsigned int status;
};

// Up to NT rows of x, all of them in each CTA. Stages fill 96 KB, so that two CTAs share an SM and one's first loads run under the other's last
// sums.
template <int NT>
struct Narrow {
  static constexpr uint32_t kW = 128 * 128;
  static constexpr uint32_t kX = NT * 128;
  static constexpr uint32_t kStage = kW + kX;
  static constexpr int kStages = 98304 / kStage;
  static constexpr uint32_t kOffMisc = kStages * kStage;
  static constexpr size_t kSmem = kOffMisc + sizeof(NarrowMisc) + 1024;
  static_assert(kStages <= 16 && NT * 128 * 4 <= kOffMisc, "");
};

// PARTS: CTAs of the cluster, which share K.
template <int NT, int PARTS>
__global__ void __launch_bounds__(kNarrowThreads)
    gemm_narrow_kernel(const __grid_constant__ GemmParams P, const __grid_constant__ CUtensorMap x_map,
                       const __grid_constant__ CUtensorMap w_map) {
  using C = Narrow<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  NarrowMisc* misc = reinterpret_cast<NarrowMisc*>(smem + C::kOffMisc);
  volatile int* abort_flag = &misc->abort;
  unsigned int* status = P.status != nullptr ? P.status : &misc->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_addr(&misc->full[s]), 1);
      mbar_init(smem_addr(&misc->empty[s]), 1);
    }
    mbar_init(smem_addr(&misc->acc_full), 1);
    misc->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&x_map);
    tma_prefetch_desc(&w_map);
  }
  constexpr uint32_t kCols = NT < 32 ? 32 : NT;
  if (warp == 1) {
    tmem_alloc(smem_addr(&misc->tmem_base), kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  pdl_wait();
  const uint32_t tmem = misc->tmem_base;
  const int f0 = static_cast<int>(blockIdx.x) / PARTS * 128;  // (all rows of x are one tile)
  const int k0 = static_cast<int>(static_cast<int64_t>(P.k_blocks) * rank / PARTS);
  const int k1 = static_cast<int>(static_cast<int64_t>(P.k_blocks) * (rank + 1) / PARTS);

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      for (int k = k0; k < k1; ++k, ++it) {
        const int s = it % C::kStages;
        if (it >= C::kStages && !wait_bar(smem_addr(&misc->empty[s]), (it / C::kStages - 1) & 1, abort_flag, status))
          break;
        const uint32_t full = smem_addr(&misc->full[s]);
        mbar_arrive_expect_tx(full, C::kStage);
        tma_load_2d(sb + s * C::kStage, &w_map, 64 * k, f0, full);
        tma_load_2d(sb + s * C::kStage + C::kW, &x_map, 64 * k, 0, full);
      }
      if (*abort_flag)
        for (int k = 1; k <= C::kStages && it - k >= 0; ++k)
          mbar_wait_drain(smem_addr(&misc->full[(it - k) % C::kStages]), ((it - k) / C::kStages) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, NT, 0, 0);
      const uint64_t kmaj = sdesc_sw128(0, 16, 1024);
      int it = 0;
      for (int k = k0; k < k1; ++k, ++it) {
        const int s = it % C::kStages;
        if (!wait_bar(smem_addr(&misc->full[s]), (it / C::kStages) & 1, abort_flag, status)) break;
        tc_fence_after();
        const uint64_t a = kmaj | ((sb + s * C::kStage) >> 4);
        const uint64_t b = kmaj | ((sb + s * C::kStage + C::kW) >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_bf16_ss(tmem, a + 2 * i, b + 2 * i, idesc, (it | i) ? 1u : 0u);
        mma_commit(smem_addr(&misc->empty[s]));
      }
      mma_commit(smem_addr(&misc->acc_full));
    }
  } else {
    // this CTA's sums to its own shared memory [row of x][feature] (the stages are free: every product has completed)
    const int quarter = warp & 3;
    const bool ok = wait_bar(smem_addr(&misc->acc_full), 0, abort_flag, status);
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < NT; c += 16) {
      uint32_t r[16];
      tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, r);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        reinterpret_cast<float*>(smem)[(c + i) * 128 + quarter * 32 + lane] =
            ok && k1 > k0 ? __uint_as_float(r[i]) : 0.f;
    }
    tc_fence_before();
  }
  __syncthreads();
  // TMEM goes before the peers are waited for: where this SM's or a peer's holds blocks of another kernel that want TMEM too,
  // nobody waits for columns of a CTA that itself waits for one without
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
  cluster_sync_all();
  // Rank r sums and writes every PARTS-th row: a warp a row, four features a lane; its loads from the peers (and of the
  // residual) are in flight together.
  constexpr int kWarps = kNarrowThreads / 32, kAtOnce = 16 / PARTS;
  const int f = 4 * lane;
  const bool inside = f0 + f < P.cols;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (P.bias != nullptr && inside) {
    const uint2 b = *reinterpret_cast<const uint2*>(P.bias + f0 + f);
    bias[0] = __uint_as_float(b.x << 16);
    bias[1] = __uint_as_float(b.x & 0xFFFF0000u);
    bias[2] = __uint_as_float(b.y << 16);
    bias[3] = __uint_as_float(b.y & 0xFFFF0000u);
  }
  for (int i0 = warp * PARTS + rank; i0 < P.rows; i0 += kAtOnce * kWarps * PARTS) {
    float4 y[kAtOnce];
    uint2 res[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kWarps * PARTS;
      res[u] = make_uint2(0, 0);
      if (P.residual != nullptr && i < P.rows && inside)
        res[u] = *reinterpret_cast<const uint2*>(P.residual + i * P.residual_stride + f0 + f);
    }
    float4 v[PARTS][kAtOnce];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      const uint32_t peer = map_shared_rank(sb + f * 4, p);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int i = i0 + u * kWarps * PARTS;
        v[p][u] = i < P.rows ? ld_shared_cluster_v4(peer + i * 512) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      y[u] = v[0][u];
#pragma unroll
      for (int p = 1; p < PARTS; ++p) {
        y[u].x += v[p][u].x;
        y[u].y += v[p][u].y;
        y[u].z += v[p][u].z;
        y[u].w += v[p][u].w;
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kWarps * PARTS;
      if (i >= P.rows || !inside) continue;
      float v[4] = {y[u].x + bias[0], y[u].y + bias[1], y[u].z + bias[2], y[u].w + bias[3]};
      if (P.act != kPlain) {
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const float2 x = make_float2(v[k], v[k + 1]);
          const float2 a = P.act == kSilu ? activate<kSilu>(x) : activate<kGelu>(x);
          v[k] = a.x;
          v[k + 1] = a.y;
        }
      }
      if (P.residual != nullptr) {
        v[0] += __uint_as_float(res[u].x << 16);
        v[1] += __uint_as_float(res[u].x & 0xFFFF0000u);
        v[2] += __uint_as_float(res[u].y << 16);
        v[3] += __uint_as_float(res[u].y & 0xFFFF0000u);
      }
      *reinterpret_cast<uint2*>(P.out + i * P.out_stride + f0 + f) =
          make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
    }
  }
  cluster_sync_all();  // no CTA leaves while a peer reads its sums
}

template <int NT, int PARTS>
cudaError_t narrow(const GemmParams& p, const CUtensorMap& x_map, const CUtensorMap& w_map, int grid, cudaStream_t stream) {
  auto kern = gemm_narrow_kernel<NT, PARTS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Narrow<NT>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kNarrowThreads);
  cfg.dynamicSmemBytes = Narrow<NT>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = PARTS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p, x_map, w_map);
}

template <int NT>
cudaError_t narrow_by(const GemmParams& p, const CUtensorMap& x_map, const CUtensorMap& w_map, int grid, cudaStream_t stream) {
  switch (p.split) {
    case 1: return narrow<NT, 1>(p, x_map, w_map, grid, stream);
    case 2: return narrow<NT, 2>(p, x_map, w_map, grid, stream);
    case 4: return narrow<NT, 4>(p, x_map, w_map, grid, stream);
    default: return narrow<NT, 8>(p, x_map, w_map, grid, stream);
  }
}

}  // namespace

cudaError_t launch_gemm_pair(const GemmParams& p, const CUtensorMap& x_map, const CUtensorMap& w_map,
                             const CUtensorMap& y_map, int clusters, cudaStream_t stream) {
  auto go = [&](auto kern) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(2 * clusters), dim3(kGemmThreads), kGemmSmem, stream, p, x_map, w_map, y_map);
  };
  if (p.value_wide != nullptr) return go(gemm_pair_kernel<kKeysValues>);
  return p.act == kPlain ? go(gemm_pair_kernel<kPlain>) : p.act == kSilu ? go(gemm_pair_kernel<kSilu>) : go(gemm_pair_kernel<kGelu>);
}

cudaError_t launch_gemm_narrow(int rows_a_cta, const GemmParams& p, const CUtensorMap& x_map, const CUtensorMap& w_map,
                               int grid, cudaStream_t stream) {
  switch (rows_a_cta) {
    case 16: return narrow_by<16>(p, x_map, w_map, grid, stream);
    case 32: return narrow_by<32>(p, x_map, w_map, grid, stream);
    case 64: return narrow_by<64>(p, x_map, w_map, grid, stream);
    default: return narrow_by<128>(p, x_map, w_map, grid, stream);
  }
}

}  // namespace mla
