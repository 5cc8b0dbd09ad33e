// Paged-latent MLA decode over 4-bit rows (MLA_KV_FP4_448_UE8M0, MLA_KV_FP4_512_UE8M0) on CTA pairs (sm_103a), for
// query rows in groups of 128 (heads x draft tokens, e.g. 128 heads), dense or over listed rows.
//
// The same computation as decode_sm103.cu ("mla_attention.py · tduncan/Nvidia-Optimization-Stack-VLLM",
// module docstring, "Data-Movement Friendly Approach"), on the pair schedule of decode_pair_sm103.cu: a
// cluster of two CTAs takes 128 query rows, CTA c the query rows 64c .. 64c + 63 and, of every 128-row KV tile,
// rows 64c .. 64c + 63.
//   S = Q K^T   M = 128 (64 query rows a CTA) x N = 128 KV rows (64 from each CTA's shared memory); lane
//               r + 64h, column n of a CTA's accumulator is its query row r against KV row n of tile half h.
//   O += P V    M = 128 x N = 256 value dims (128 from each CTA) x K = 128 KV rows, two blocks b; lane
//               r + 64h, column 128b + d is dim 256b + 128h + d of query row r.
// What differs is where the operands come from. Nothing of a 4-bit row can be copied to shared memory as it
// is: eight converter warps a CTA write its 64 rows as bf16 (all dims: the S operand), and, into the slabs
// that S has read and this CTA's half of V does not need, the peer's 64 rows in this CTA's 256 value dims.
// That is three conversions of a half row for two SMs' work, against four (two whole rows) when the groups run
// on one SM each, and S runs at N = 128 instead of M = 64. Measured against the single-SM kernel, us, 128 heads:
//   64 requests, 295K rows in all            116 (708 TFLOP/s)   156
//   32 requests x 4 draft tokens             389 (846 TFLOP/s)   552
//   2048 listed rows for each of 64 tokens    66                  84
//   one request of 131071 rows                64 (59 and the merge of 76 partials)
// A tile takes about 5.7K cycles, of which the tensor cores work 2.8K (36 S steps of 49 cycles, 16 PV steps of 64).
// They are a chain: with two stages, the operand of S(t + 1) waits for the values of tile t, those for S(t), and S(t)
// for its operand (traced: 0.6K cycles from S to its values, 2K to the operand's first part, 3.4K of S and the PV
// between). What it holds to: no load waited for soon after its issue (each row's address runs three tiles ahead, RoPE
// goes past the registers), few instructions a group of codes and an MMA (issue slots are 45% used, the issuers share
// theirs with four busy warps), and code that stays small beside the instruction cache.
//
// Shared memory per CTA: Q (64 rows x 64 dims a slab, 128-B swizzle), two stages of the tile's rows, P of the
// tile's two halves: the 512-NoPE row's P of half 0 takes its stage's RoPE slab, which V does not read and S
// has read; the 448-NoPE row has eight slabs, all of them V, and two P slabs beside.
//
// Warp roles (640 threads):
//   warp 0       Q by TMA once per unit
//   warp 1       TMEM allocation; L2 prefetch of the tile after next (dense)
//   warp 2       S MMA issuer (even CTA only)
//   warp 3       PV MMA issuer (even CTA only)
//   warps 4-11   softmax (lane r + 64h: query row r over tile half h; warps 4-7 take S columns 0-31 and
//                O block 0, warps 8-11 columns 32-63 and O block 1), O rescale, epilogue
//   warps 12-19  converters: 8 rows of each tile half a warp
#include <cstdint>
#include <cuda_runtime.h>

#include "decode_common.cuh"
#include "kv_row.cuh"
#include "mla_kernels.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

constexpr int kPairThreads = 640;
constexpr uint32_t kPSlab = 8192;  // 64 rows x 128 B
constexpr float kPairRescaleLog2 = 64.0f;  // as the single-SM kernel: P, O and the sums stay inside fp32

template <int LAYOUT>
struct Cfg {
  static constexpr int kNope = row_nope(LAYOUT);
  static constexpr int kNslab = row_width(LAYOUT) / 64;
  static constexpr int kRowBytes = row_stored_bytes(LAYOUT);
  // A tile's S operand arrives in parts: slabs 0-3, slabs 4-7 (with the RoPE slab as the eighth of the 448-NoPE
  // row), and the RoPE slab of the 512-NoPE row.
  static constexpr int kParts = kNslab == 9 ? 3 : 2;
  static constexpr uint32_t kOffStage = kNslab * kPSlab;
  static constexpr uint32_t kStageBytes = kNslab * kPSlab;
  static constexpr uint32_t kOffP = kOffStage + 2 * kStageBytes;  // P of half 1, and of half 0 for eight slabs
  static constexpr uint32_t kOffMisc = kOffP + (kNslab == 9 ? 1 : 2) * kPSlab;
};

// Every barrier whose arrivals for tile t + 1 could come before its waiter has seen tile t
// is kept per stage (or per TMEM buffer): a parity wait must never be more than one phase
// behind.
enum PairBar {
  // gates of the MMA issuers, arrived on from both CTAs (used in the even CTA)
  kQFull = 0,       // count 2, + bytes
  kSRegFull = 1,    // + 3 * stage + part (2 x 3): count 16 (the converter warps of both CTAs)
  kPFull = 7,       // count 16 (the softmax warps of both CTAs)
  kSFree = 8,       // + TMEM buffer (2): count 16
  kOFree = 10,      // count 16
  // signalled in both CTAs by the even CTA's multicast commits
  kSFull = 11,      // + TMEM buffer (2)
  kSDone = 13,      // + 4 * stage + 2 * b + h (2 x 4): S has read the slabs 4b + 2h + {0, 1}
  kStageFree = 21,  // + stage (2): the PV of the stage's tile has completed
  kPvDone = 23,
  kQEmpty = 24,
  kOFull = 25,
  // local to each CTA
  kVFull = 26,      // + stage (2): count 8 (converter warps): the peer rows' values
  kMask = 28,       // + stage (2): count 8: which rows of the tile count
  kFinal = 30,      // count 2: the last commit of each issuer (even CTA)
  kNumPairBars = 31
};

struct PairMisc {
  uint64_t bar[kNumPairBars];
  uint32_t tmem_base;
  int abort;
  int progress;            // tiles whose conversion has begun (throttles the prefetch)
  int pad;
  uint8_t mask[2][16];      // per stage, 8 rows each: tile half 0's rows, then half 1's
  // the four threads of a query row exchange their tile maxima (slow path of a tile) and,
  // at the end of a unit, their partial sums here
  float xchg[256];
};
static_assert(Cfg<4>::kOffMisc + sizeof(PairMisc) + 1024 <= 232448, "shared memory budget of one CTA");
static_assert(Cfg<3>::kOffMisc + sizeof(PairMisc) + 1024 <= 232448, "shared memory budget of one CTA");

// mma_bf16_pair with the operands' descriptors given by their low words (the start address; an offset within shared
// memory does not carry out of it): half the arithmetic of an MMA in the issuers, whose instructions wait their turn
// among the other roles' (125 us against 128; PV held back behind the next tile's S instead: 132).
__device__ __forceinline__ void mma_bf16_pair_lo(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// (a.x, a.y) * (b, b) + (c.x, c.y), and a + b, two lanes an instruction
__device__ __forceinline__ float2 fma2(float2 a, float b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 p, q, s, d;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %4};\n mov.b64 s, {%5, %6};\n"
      " fma.rn.f32x2 d, p, q, s;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 p, q, d;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n add.rn.f32x2 d, p, q;\n"
      " mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// 16 bytes of global memory to shared memory, past the registers; zeros where `on` is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// One group of 32 codes with a scale that f16 does not hold, chunk q to addr ^ (q << 4); out of line, for it is rare.
__device__ __noinline__ void put_wide(uint4 v, uint32_t sbyte, uint32_t addr) {
  const Fp4Scale s = fp4_scale(sbyte);
  const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t e[4];
    fp4x8_to_bf16(w4[q], s, e);
    st_shared_v4(addr ^ (q << 4), make_uint4(e[0], e[1], e[2], e[3]));
  }
}

// Predicated loads (no branch): zeros, or `other`, where `on` is false. (Not the non-coherent ones: this grid may be on
// its SMs before the grid that writes the rows has ended.)
__device__ __forceinline__ uint4 ld_or_zero(const void* p, bool on) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n mov.u32 %3, 0;\n"
      " @p ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(static_cast<uint32_t>(on)));
  return v;
}
// The same of 32 bytes (32-byte aligned), in one load: two of 16 would ask for every sector twice.
__device__ __forceinline__ void ld32_or_zero(const void* p, bool on, uint4& a, uint4& b) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %9, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n mov.u32 %3, 0;\n"
      " mov.u32 %4, 0;\n mov.u32 %5, 0;\n mov.u32 %6, 0;\n mov.u32 %7, 0;\n"
      " @p ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n}\n"
      : "=&r"(a.x), "=&r"(a.y), "=&r"(a.z), "=&r"(a.w), "=&r"(b.x), "=&r"(b.y), "=&r"(b.z), "=&r"(b.w)
      : "l"(p), "r"(static_cast<uint32_t>(on)));
}
__device__ __forceinline__ int ld_i32_or(const int32_t* p, bool on, int other) {
  int v;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.s32 %0, %3;\n @p ld.global.s32 %0, [%1];\n}\n"
               : "=&r"(v)
               : "l"(p), "r"(static_cast<uint32_t>(on)), "r"(other));
  return v;
}
__device__ __forceinline__ uint32_t ld_u16_or(const void* p, bool on, uint32_t other) {
  uint32_t v;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.u32 %0, %3;\n @p ld.global.u16 %0, [%1];\n}\n"
               : "=&r"(v)
               : "l"(p), "r"(static_cast<uint32_t>(on)), "r"(other));
  return v;
}
__device__ __forceinline__ uint32_t ld_u8_or(const void* p, bool on, uint32_t other) {
  uint32_t v;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.u32 %0, %3;\n @p ld.global.u8 %0, [%1];\n}\n"
               : "=&r"(v)
               : "l"(p), "r"(static_cast<uint32_t>(on)), "r"(other));
  return v;
}

template <int LAYOUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mla_decode_pair_fp4_kernel(const __grid_constant__ DecodeParams P, const __grid_constant__ CUtensorMap q_map) {
  using C = Cfg<LAYOUT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  PairMisc* misc = reinterpret_cast<PairMisc*>(smem + C::kOffMisc);
  auto bar = [&](int i) -> uint32_t { return smem_addr(&misc->bar[i]); };
  volatile int* abort_flag = &misc->abort;
  auto stage = [&](int st) -> uint32_t { return sb + C::kOffStage + st * C::kStageBytes; };

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int c = static_cast<int>(rank);
  const bool leader = rank == 0;
  // P of tile half h
  auto parea = [&](int st, int h) -> uint32_t {
    if (C::kNslab == 9) return h ? sb + C::kOffP : stage(st) + 8 * kPSlab;
    return sb + C::kOffP + h * kPSlab;
  };
  const int32_t* const runs = P.runs;
  const bool sparse = P.indices != nullptr || runs != nullptr;
  auto lead = [&](int i) -> uint32_t { return map_shared_rank(bar(i), 0); };  // the even CTA's barrier

  if (tid == 0) {
    mbar_init(bar(kQFull), 2);
    for (int s = 0; s < 6; ++s) mbar_init(bar(kSRegFull + s), 16);
    mbar_init(bar(kPFull), 16);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kSFree + s), 16);
      mbar_init(bar(kSFull + s), 1);
      mbar_init(bar(kStageFree + s), 1);
      mbar_init(bar(kVFull + s), 8);
      mbar_init(bar(kMask + s), 8);
      for (int g = 0; g < 4; ++g) mbar_init(bar(kSDone + 4 * s + g), 1);
    }
    mbar_init(bar(kOFree), 16);
    mbar_init(bar(kPvDone), 1);
    mbar_init(bar(kQEmpty), 1);
    mbar_init(bar(kOFull), 1);
    mbar_init(bar(kFinal), 2);
    misc->abort = 0;
    misc->progress = 0;
    fence_mbar_init();
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
  const uint32_t tmem_o = tmem;        // O: 2 blocks x 128 columns
  const uint32_t tmem_s = tmem + 256;  // S: 2 buffers x 64 columns

  const int R = P.rows_per_req;
  const int PG = R >> 7;  // groups of 128 query rows per request
  const int num_work = P.num_partitions * PG;
  const int cl0 = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(num_clusters_x());
  // Registers: 640 threads x 96 at launch; the issuing warps give some of theirs to the softmax, which spilled with 96
  // (64 and 112 instead of 72 and 104: 396 us against 393 on the draft tokens above).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // ------------------------------------------------------------ queries
      if (lane == 0) {
        tma_prefetch_desc(&q_map);
        int u = 0;
        for (int w = cl0; w < num_work && !*abort_flag; w += ncl) {
          const int part = w / PG, g = w % PG;
          for_each_unit(P, part, [&](int r, int, int, int) {
            if (*abort_flag) return;
            if (u > 0 && !wait_bar(bar(kQEmpty), (u - 1) & 1, abort_flag, P.status)) return;
            mbar_arrive_expect_tx_cluster(lead(kQFull), C::kNslab * kPSlab);
            const int row0 = r * R + g * 128 + 64 * c;
            for (int s = 0; s < C::kNslab; ++s) tma_load_2d_pair(sb + s * kPSlab, &q_map, s * 64, row0, lead(kQFull));
            ++u;
          });
        }
        // copies still in flight land on the even CTA's gate: wait for them (bounded)
        if (*abort_flag && leader && u > 0) mbar_wait_drain_cluster(bar(kQFull), (u - 1) & 1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ L2 prefetch (dense)
      // This CTA's rows of coming tiles, and their scale slots, into L2: two tiles ahead of the conversion, a page's
      // part at a time (one lane each). A hint: nothing waits on it.
      if (!sparse) {
        const int box = P.page_size < kBlockRows ? P.page_size : kBlockRows;
        int pit = 0;
        for (int w = cl0; w < num_work && !*abort_flag; w += ncl) {
          const int part = w / PG;
          for_each_unit(P, part, [&](int r, int lo, int hi, int) {
            if (*abort_flag) return;
            const int L = request_len(P, r);
            for (int b0 = lo; b0 < hi; b0 += 2, ++pit) {
              const uint64_t t0 = globaltimer();
              while (pit >= *reinterpret_cast<volatile int*>(&misc->progress) + 3) {
                if (*abort_flag) return;
                if (globaltimer() - t0 > 20000000ull) break;  // stop throttling after 20 ms
                __nanosleep(200);
              }
              const int blk = b0 + c;
              for (int pos0 = blk * kBlockRows + lane * box; blk < hi && pos0 < (blk + 1) * kBlockRows && pos0 < L;
                   pos0 += 32 * box) {
                const int pi = pos0 >> P.log2_ps;
                const int page = pi < P.max_pages ? P.block_table[static_cast<int64_t>(r) * P.max_pages + pi] : -1;
                if (page < 0 || page >= P.num_pages) continue;
                const int off = pos0 & (P.page_size - 1);
                const int rows = L - pos0 < box ? L - pos0 : box;
                const uint8_t* pg = P.kv + static_cast<int64_t>(page) * P.page_bytes;
                prefetch_l2_bulk(pg + static_cast<int64_t>(off) * C::kRowBytes, rows * C::kRowBytes);
                prefetch_l2_bulk(pg + static_cast<int64_t>(P.page_size) * C::kRowBytes + off * kFp4ScaleSlot,
                                 rows * kFp4ScaleSlot);
              }
            }
          });
        }
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ S issuer (even CTA)
      if (leader && lane == 0) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);
        const uint64_t kmaj = sdesc_sw128(0, 16, 1024);
        const uint32_t khi = static_cast<uint32_t>(kmaj >> 32);
        const uint32_t qa = static_cast<uint32_t>(kmaj) | (sb >> 4);
        int it = 0, u = 0;
        for (int w = cl0; w < num_work && !*abort_flag; w += ncl) {
          const int part = w / PG;
          for_each_unit(P, part, [&](int, int lo, int hi, int) {
            if (*abort_flag) return;
            if (!wait_bar(bar(kQFull), u & 1, abort_flag, P.status)) return;
            for (int b0 = lo; b0 < hi; b0 += 2, ++it) {
              const int st = it & 1;
              if (it >= 2 && !wait_bar(bar(kSFree + st), ((it >> 1) - 1) & 1, abort_flag, P.status)) return;
              tc_fence_after();
              const uint32_t d = tmem_s + st * 64;
              const uint32_t ka = static_cast<uint32_t>(kmaj) | (stage(st) >> 4);
              // Fully unrolled, so that the descriptors are the base plus constants: an MMA issued
              // from a loop that computes its descriptors costs about 70 cycles, unrolled about 50.
#pragma unroll
              for (int s = 0; s < C::kNslab; ++s) {
                if ((s & 3) == 0) {
                  if (!wait_bar(bar(kSRegFull + 3 * st + (s >> 2)), (it >> 1) & 1, abort_flag, P.status)) return;
                  tc_fence_after();
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_bf16_pair_lo(d, qa + s * (kPSlab >> 4) + kk * 2, khi, ka + s * (kPSlab >> 4) + kk * 2, khi,
                                   idesc_s, (s | kk) ? 1u : 0u);
                // value slabs 4b + 2h + {0, 1} read: the peer rows' values may overwrite them
                if (s < 8 && (s & 1)) mma_commit_pair(bar(kSDone + 4 * st + (s >> 1)), 3);
              }
              // (failure-detection test: withhold the first tile's signal so that the
              // softmax's bounded wait runs out)
              if (!(P.test_withhold_signal && it == 0)) mma_commit_pair(bar(kSFull + st), 3);
            }
            mma_commit_pair(bar(kQEmpty), 3);
            ++u;
          });
        }
        mma_commit_pair(bar(kFinal), 1);
        mbar_wait_drain_cluster(bar(kFinal), 0);
      }
    } else if (warp == 3) {
      // ------------------------------------------------------------ PV issuer (even CTA)
      if (leader && lane == 0) {
        constexpr uint32_t idesc_o = idesc_bf16_f32(128, 256, 0, 1);  // A = P (K-major), B = V (MN-major)
        const uint64_t kmaj = sdesc_sw128(0, 16, 1024);
        const uint64_t vmaj = sdesc_sw128(0, kPSlab, 1024);
        const uint32_t phi = static_cast<uint32_t>(kmaj >> 32), vhi = static_cast<uint32_t>(vmaj >> 32);
        int it = 0, u = 0;
        for (int w = cl0; w < num_work && !*abort_flag; w += ncl) {
          const int part = w / PG;
          for_each_unit(P, part, [&](int, int lo, int hi, int) {
            if (*abort_flag) return;
            for (int b0 = lo; b0 < hi; b0 += 2, ++it) {
              const int st = it & 1;
              const bool first = b0 == lo;
              if (!wait_bar(bar(kPFull), it & 1, abort_flag, P.status)) return;
              if (first && u > 0 && !wait_bar(bar(kOFree), (u - 1) & 1, abort_flag, P.status)) return;
              tc_fence_after();
              const uint32_t p0 = static_cast<uint32_t>(kmaj) | (parea(st, 0) >> 4);
              const uint32_t p1 = static_cast<uint32_t>(kmaj) | (parea(st, 1) >> 4);
              const uint32_t vb = static_cast<uint32_t>(vmaj) | (stage(st) >> 4);
#pragma unroll
              for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const int h = k >> 2;
                  const uint32_t a = (h ? p1 : p0) + (k & 3) * 2;
                  const uint32_t bv = vb + (4 * b + 2 * h) * (kPSlab >> 4) + (k & 3) * (2048 >> 4);
                  mma_bf16_pair_lo(tmem_o + b * 128, a, phi, bv, vhi, idesc_o, (first && k == 0) ? 0u : 1u);
                }
              }
              mma_commit_pair(bar(kPvDone), 3);
              mma_commit_pair(bar(kStageFree + st), 3);
            }
            mma_commit_pair(bar(kOFull), 3);
            ++u;
          });
        }
        mma_commit_pair(bar(kFinal), 1);
        mbar_wait_drain_cluster(bar(kFinal), 0);
      }
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ------------------------------------------------------------ softmax / epilogue
    // Lane wt = r + 64h of TMEM holds query row r (of this CTA's 64) against KV tile half
    // h in S, and dims 256b + 128h + 0..127 of that row in O. Two warps share each
    // 32-lane quarter (a warp reaches the lanes 32 (warp % 4) .. + 31): column group
    // cg = 0 takes S columns 0-31 and O block 0, cg = 1 columns 32-63 and O block 1. The
    // four threads of a row meet through shared memory; the four warps that hold the same 32
    // rows meet at a named barrier of theirs (all eight at one: 1% slower; no time limit: a
    // thread whose bounded wait fails marks itself dead and all stop together at the next
    // barrier, the other four warps when the abort ends a wait of theirs).
    const int sx = tid - 128;  // 0 .. 255
    const int cg = sx >> 7;
    const int wt = sx & 127;
    const int r = wt & 63;
    const int half = wt >> 6;
    const int rows_bar = 1 + (warp & 1);  // of the four warps that share query rows 32 (warp % 2) .. + 31
    const uint32_t lane_off = static_cast<uint32_t>(wt & ~31) << 16;
    bool dead = false, stop = false;
    auto wait = [&](uint32_t b, uint32_t parity) {
      if (!dead && !wait_bar(b, parity, abort_flag, P.status)) dead = true;
      return !dead;
    };
    int it = 0, u = 0;
    for (int w = cl0; w < num_work && !stop; w += ncl) {
      const int part = w / PG, g = w % PG;
      const int grow = g * 128 + 64 * c + r;  // query row within the request
      const int tok = grow / P.heads;
      for_each_unit(P, part, [&](int rq, int lo, int hi, int sidx) {
        if (stop) return;
        // causal: KV positions < row_end count for this query row
        const int row_end = P.causal && !sparse ? request_len(P, rq) - P.sq + tok + 1 : 0x7fffffff;
        float m_run = -INFINITY, l_run = 0.f;
        for (int b0 = lo; b0 < hi; b0 += 2, ++it) {
          const int st = it & 1;
          const bool first = b0 == lo;
          uint32_t sr[32];
          wait(bar(kMask + st), (it >> 1) & 1);
          const uint32_t held = *reinterpret_cast<const uint32_t*>(&misc->mask[st][8 * half + 4 * cg]);
          wait(bar(kSFull + st), (it >> 1) & 1);
          if (!dead) {
            tc_fence_after();
            tmem_ld32(tmem_s + st * 64 + lane_off + cg * 32, sr);
            tmem_wait_ld();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(lead(kSFree + st));
          const int pos0 = (b0 + half) * kBlockRows + cg * 32;  // KV position of this thread's column 0
          int nv = row_end - pos0;
          nv = nv < 0 ? 0 : (nv > 32 ? 32 : nv);
          const uint32_t vmask = held & (nv == 32 ? ~0u : ((1u << nv) - 1u));
          // masked scores become -inf: weight 0 (rarely any: one test a warp)
          if (!__all_sync(0xffffffffu, vmask == ~0u)) {
#pragma unroll
            for (int cc = 0; cc < 32; ++cc) sr[cc] = ((vmask >> cc) & 1u) ? sr[cc] : 0xFF800000u;
          }
          float mt0 = -INFINITY, mt1 = -INFINITY;
#pragma unroll
          for (int cc = 0; cc < 32; cc += 4) {
            mt0 = max3(mt0, __uint_as_float(sr[cc]), __uint_as_float(sr[cc + 1]));
            mt1 = max3(mt1, __uint_as_float(sr[cc + 2]), __uint_as_float(sr[cc + 3]));
          }
          const float mt = fmaxf(mt0, mt1) * P.scale_log2;
          // the running maximum of a row moves (lazily) only when a tile exceeds it by more
          // than kPairRescaleLog2 powers of two; the four threads of the row take the same
          // decision
          const bool raise = mt > m_run + kPairRescaleLog2;
          float m_new = m_run;
          const bool any = named_bar_or(rows_bar, 128, raise || dead);
          if (any) {
            if (named_bar_or(rows_bar, 128, dead)) {
              stop = true;
              return;
            }
            misc->xchg[sx] = mt;
            named_bar_sync(rows_bar, 128);
            const float mh = fmaxf(fmaxf(misc->xchg[r], misc->xchg[r + 64]),
                                   fmaxf(misc->xchg[128 + r], misc->xchg[128 + r + 64]));
            m_new = (mh > m_run + kPairRescaleLog2) ? mh : m_run;
          }
          const bool rescale = any && !first && m_new != m_run && m_run != -INFINITY;
          const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
          const float alpha = fast_exp2(m_run - m_use);
          float2 ps = make_float2(0.f, 0.f);
          uint32_t pk[16];
#pragma unroll
          for (int cc = 0; cc < 16; ++cc) {
            const float2 x = fma2(make_float2(__uint_as_float(sr[2 * cc]), __uint_as_float(sr[2 * cc + 1])),
                                  P.scale_log2, make_float2(-m_use, -m_use));
            const float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            ps = add2(ps, p);
            pk[cc] = f32x2_to_bf16x2(p.x, p.y);
          }
          l_run = l_run * alpha + (ps.x + ps.y);
          m_run = m_new;
          // P and O belong to the previous tile's PV until it completes
          if (it > 0) wait(bar(kPvDone), (it - 1) & 1);
          if (any && !first && !dead) {
            // one TMEM round trip per 32 columns of this thread's 128 O columns
            tc_fence_after();
            const float a = rescale ? alpha : 1.0f;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              uint32_t t32[32];
              const uint32_t ta = tmem_o + lane_off + cg * 128 + k * 32;
              tmem_ld32(ta, t32);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) t32[i] = __float_as_uint(__uint_as_float(t32[i]) * a);
              tmem_st32(ta, t32);
            }
            tmem_wait_st();
            tc_fence_before();
          }
          if (!dead) {
            // P row r: KV rows of tile half `half`, 64 bf16 along K (K-major, 128-B swizzle),
            // of which this thread holds the 16-B chunks 4 cg .. 4 cg + 3
            const uint32_t pa = parea(st, half) + r * 128;
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
              st_shared_v4(pa + (((4 * cg + q4) ^ (r & 7)) << 4),
                           make_uint4(pk[4 * q4], pk[4 * q4 + 1], pk[4 * q4 + 2], pk[4 * q4 + 3]));
          }
          wait(bar(kVFull + st), (it >> 1) & 1);  // the peer rows' values are in place
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && !dead) mbar_arrive_cluster(lead(kPFull));
        }
        // -------------------------------------------------------- epilogue
        named_bar_sync(rows_bar, 128);  // every thread has read the last tile's maxima
        misc->xchg[sx] = l_run;
        if (named_bar_or(rows_bar, 128, dead)) {
          stop = true;
          return;
        }
        const float l_tot = (misc->xchg[r] + misc->xchg[r + 64]) + (misc->xchg[128 + r] + misc->xchg[128 + r + 64]);
        const int base_split = P.num_splits[rq];
        const int nsplit = P.num_splits[rq + 1] - base_split;
        const int sg = base_split + sidx;
        float inv = 0.f, lse2 = -INFINITY;
        if (!(l_tot <= 0.f)) {  // a NaN sum, from a NaN group, is passed on
          float denom = l_tot;
          if (nsplit == 1 && P.sink != nullptr)
            denom += fast_exp2(P.sink[grow % P.heads] * 1.4426950408889634f - m_run);
          inv = 1.0f / denom;
          lse2 = m_run + log2f(l_tot);
        }
        if (half == 0 && cg == 0) {
          const float lse_nat = lse2 * 0.6931471805599453f;
          if (nsplit == 1) P.lse[(int64_t)rq * R + grow] = lse_nat;
          else P.part_lse[(int64_t)sg * R + grow] = lse_nat;
        }
        if (wait(bar(kOFull), u & 1)) {
          tc_fence_after();
          // A warp holds 32 consecutive output rows (one per lane) and, per TMEM load, the same
          // 32 value dims of each. Eight rows at a time pass through this warp's 1-KiB slice of
          // the P slab (free here: the unit's last PV has completed, and the next P of the slice's rows is
          // written by warps of this one's barrier; 16-B chunk q of staged row i
          // at position q ^ i), so that each global store covers contiguous dims of one row
          // (a store of one 16-B chunk per lane would touch 32 rows).
          const uint32_t xb = parea(0, 1) + static_cast<uint32_t>((warp & 1) * 4 + ((warp - 4) >> 1)) * 1024u;
          const int64_t row0 = (nsplit == 1 ? (int64_t)rq : (int64_t)sg) * R + (grow - lane);
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t t32[32];
            tmem_ld32(tmem_o + lane_off + cg * 128 + k * 32, t32);
            tmem_wait_ld();
            const int d0 = cg * 256 + half * 128 + k * 32;  // first value dim of these 32 columns
#pragma unroll
            for (int rnd = 0; rnd < 4; ++rnd) {
              if ((lane >> 3) == rnd) {
                const uint32_t i = static_cast<uint32_t>(lane & 7);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  st_shared_v4(xb + i * 128 + ((static_cast<uint32_t>(q) ^ i) << 4),
                               make_uint4(__float_as_uint(__uint_as_float(t32[4 * q]) * inv),
                                          __float_as_uint(__uint_as_float(t32[4 * q + 1]) * inv),
                                          __float_as_uint(__uint_as_float(t32[4 * q + 2]) * inv),
                                          __float_as_uint(__uint_as_float(t32[4 * q + 3]) * inv)));
              }
              __syncwarp();
              if (nsplit == 1) {
                // bf16: 16 lanes per row, two dims each, two rows per store
                const int m = lane & 15;
#pragma unroll
                for (int i2 = 0; i2 < 8; i2 += 2) {
                  const uint32_t i = static_cast<uint32_t>(i2 + (lane >> 4));
                  const uint32_t at = xb + i * 128 + ((static_cast<uint32_t>(m >> 1) ^ i) << 4) + (m & 1) * 8;
                  const float2 v = ld_shared_v2f32(at);
                  reinterpret_cast<uint32_t*>(P.out + (row0 + rnd * 8 + i) * 512 + d0)[m] = f32x2_to_bf16x2(v.x, v.y);
                }
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const uint32_t at = xb + i * 128 + ((static_cast<uint32_t>(lane >> 2) ^ i) << 4) + (lane & 3) * 4;
                  P.part_out[(row0 + rnd * 8 + i) * 512 + d0 + lane] = ld_shared_f32(at);
                }
              }
              __syncwarp();
            }
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0 && !dead) mbar_arrive_cluster(lead(kOFree));
        ++u;
      });
    }
  } else {
    // ------------------------------------------------------------ converters
    // A warp takes rows 8 w .. + 7 of both tile halves (w = warp - 12), four lanes a row: of the peer's half this CTA's
    // 256 value dims (V of tile t: a group of 32 codes a lane and block), then of its CTA's own half all dims (the S
    // operand of tile t + 1: of each part a slab a lane, two groups). Lanes 0-7 look up the own half's rows, lanes 8-15
    // the peer's. Codes are loaded a conversion or more before their own (the operand's at the top of the iteration,
    // V's at the end of the one before), and every step of the address chain (listed index -> block-table entry -> row)
    // an iteration before the next: one loop body does them all, its first iterations (t < 0) only what there is. The
    // order is fixed: V(t) waits for S(t), the operand of S(t + 1) for the value product of tile t - 1, and warps that
    // each took what could go first held one another up (6% slower; the operand before the values: 4%).
    const int w8 = (warp - 12) * 8;
    const int h = 1 - c;                      // the peer's half
    const int my_half = lane < 8 ? c : h;
    const int r8 = lane & 7, g4 = lane >> 3;  // row; S operand: a slab of a part, values: a group of a block
    auto wait = [&](uint32_t b, uint32_t parity) {  // warp-uniform
      return __all_sync(0xffffffffu, wait_bar(b, parity, abort_flag, P.status));
    };
    // One group of 32 codes as four 16-byte chunks. Chunk q of the group goes to addr ^ (q << 4): addr holds the
    // row's place of chunk 0 in the 128-byte swizzle. The eight lanes that store at once hold eight rows, whose
    // places are eight different banks' groups.
    auto put = [&](uint4 v, uint32_t sbyte, uint32_t addr, bool on) {
      if (!__all_sync(0xffffffffu, fp4_scale_plain(sbyte))) {
        if (on) put_wide(v, sbyte, addr);
        return;
      }
      Fp4Scale s;
      s.h = static_cast<uint16_t>((sbyte - 112u) << 10);
      const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t e[4];
        fp4x8_to_bf16<true>(w4[q], s, e);
        if (on) st_shared_v4(addr ^ (q << 4), make_uint4(e[0], e[1], e[2], e[3]));
      }
    };
    // this thread's places (row w8 + r8): of the S operand in slab g4 of a part, of the values in slab 2h + g4 / 2, of
    // the RoPE slab
    const uint32_t row_at = (w8 + r8) * 128;
    const uint32_t own_at = g4 * kPSlab + row_at + (r8 << 4);
    const uint32_t val_at = (2 * h + (g4 >> 1)) * kPSlab + row_at + (((4 * (g4 & 1)) ^ r8) << 4);
    const uint32_t pe_at = (C::kNslab - 1) * kPSlab + row_at + ((g4 ^ r8) << 4);
    constexpr int kNopeGroups = C::kNope / kFp4Group;
    int it = 0;  // tiles whose V is in place
    bool live = true;
    for (int w = cl0; w < num_work && live; w += ncl) {
      const int part = w / PG, g = w % PG;
      for_each_unit(P, part, [&](int r, int lo, int hi, int) {
        if (!live) return;
        const int L = runs ? 0x7fffffff : request_len(P, r);
        const int tok = r * P.sq + (g * 128) / P.heads;  // listed rows: the group's token
        const int ntile = (hi - lo + 1) >> 1;
        int pos3 = -1, pos2 = -1, page2 = -1;  // this lane's row of tiles t + 3 and t + 2
        uint64_t row1 = 0;                     // address of its row of tile t + 1 (0: none)
        int32_t sc1 = 0;                       // from there to its scale slot
        // values of tile t: the two blocks' groups of the peer's row r8; where a row has eight slabs, the last
        // block's second slab is RoPE, 64 bytes a lane (16 in vr, 48 in vp)
        uint4 vr[2], vp[C::kNslab == 9 ? 1 : 3];
        uint32_t vs[2];
        uint64_t ao = 0;  // S operand of tile t + 1: this thread's row, its scales
        const uint8_t* spo = nullptr;
        uint32_t ok1 = 0;  // which rows of tile t + 1 count
        for (int t = -4; t < ntile; ++t) {
          // codes of the S operand of tile t + 1: of each part the two groups of a slab, with their scale bytes
          uint4 raw[4];
          uint32_t rs[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const bool any = ao != 0 && 8 * q + 2 * g4 < kNopeGroups;
            ld32_or_zero(reinterpret_cast<const uint8_t*>(ao) + 128 * q + 32 * g4, any, raw[2 * q], raw[2 * q + 1]);
            rs[q] = ld_u16_or(spo + 8 * q, any, 0x7F7Fu);
          }
          if (t >= 0) {
            // ---- values of tile t: the peer's rows, this CTA's dims, over slabs that S has read
            const uint32_t base = stage(it & 1);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if (!wait(bar(kSDone + 4 * (it & 1) + 2 * b + h), (it >> 1) & 1)) {
                live = false;
                return;
              }
              const bool code = 8 * b + 4 * c + g4 < kNopeGroups;
              const uint32_t at = base + 4 * b * kPSlab + val_at;
              put(vr[b], vs[b], at, code);
              if (C::kNslab == 8 && b == 1 && !code) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  st_shared_v4(at ^ (q << 4), q == 0 ? vr[1] : vp[q > 0 ? q - 1 : 0]);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kVFull + (it & 1)));
            ++it;
          }
          if (t >= -1 && t + 1 < ntile) {
            // ---- S operand of tile t + 1, whose global index `it` is by now
            const int st = it & 1;
            if (warp == 12 && lane == 0) *reinterpret_cast<volatile int*>(&misc->progress) = it + 1;
            if (it >= 2 && !wait(bar(kStageFree + st), ((it >> 1) - 1) & 1)) {
              live = false;
              return;
            }
            if (lane == 0) {
              misc->mask[st][8 * c + (w8 >> 3)] = static_cast<uint8_t>(ok1);
              misc->mask[st][8 * h + (w8 >> 3)] = static_cast<uint8_t>(ok1 >> 8);
              mbar_arrive(bar(kMask + st));
            }
            const uint32_t base = stage(st) + own_at;
            // the RoPE slab: as it is, beside the conversion
            const uint8_t* pe = (ao != 0 ? reinterpret_cast<const uint8_t*>(ao) : P.kv) + C::kNope / 2 + 16 * g4;
#pragma unroll
            for (int i = 0; i < 2; ++i) cp_async16((stage(st) + pe_at) ^ (64 * i), pe + 64 * i, ao != 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // part i / 2, group i % 2 of its slab
              put(raw[i], (rs[i >> 1] >> (8 * (i & 1))) & 0xFFu, (base + (i >> 1) * 4 * kPSlab) ^ ((i & 1) << 6),
                  8 * (i >> 1) + 2 * g4 < kNopeGroups);
              if (i == 1 || (C::kNslab == 9 && i == 3)) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(lead(kSRegFull + 3 * st + (i >> 1)));
              }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lead(kSRegFull + 3 * st + C::kParts - 1));
          }
          // ---- lookups
          uint64_t row = 0;  // of tile t + 2 (0: none)
          int32_t sc = 0;    // from there to its scale slot
          if (pos2 >= 0 && (page2 < 0 || page2 >= P.num_pages)) {  // a bad entry: the row is left out
            if (lane < 8) atomicOr(P.status, 2u);
          } else if (pos2 >= 0) {
            const int off = pos2 & (P.page_size - 1);
            row = reinterpret_cast<uint64_t>(P.kv) + (int64_t)page2 * P.page_bytes + off * C::kRowBytes;
            sc = (P.page_size - off) * C::kRowBytes + off * kFp4ScaleSlot;
            if (sparse && lane < 8) {  // rows listed one by one: each asked into L2 ahead of its load
              const uint8_t* rp = reinterpret_cast<const uint8_t*>(row);
#pragma unroll
              for (int b = 0; b < C::kRowBytes; b += 128) prefetch_l2_line(rp + b);
              prefetch_l2_line(rp + C::kRowBytes - 1);
              prefetch_l2_line(rp + sc);
            }
          }
          // ---- codes of tile t + 1's values (those of the operand follow at the top of the next iteration). All rows'
          // addresses first: a shuffle among loads in flight can come to wait for them.
          const uint64_t av = __shfl_sync(0xffffffffu, row1, 8 + r8);
          const uint8_t* spv = reinterpret_cast<const uint8_t*>(av) + __shfl_sync(0xffffffffu, sc1, 8 + r8);
          ao = __shfl_sync(0xffffffffu, row, r8);
          spo = reinterpret_cast<const uint8_t*>(ao) + __shfl_sync(0xffffffffu, sc, r8) + 2 * g4;
          ok1 = __ballot_sync(0xffffffffu, row != 0);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int gr = 8 * b + 4 * c + g4;
            const bool code = gr < kNopeGroups;
            const uint8_t* src =
                reinterpret_cast<const uint8_t*>(av) + (code ? 16 * gr : C::kNope / 2 + 64 * (gr - kNopeGroups));
            vr[b] = ld_or_zero(src, av != 0);
            vs[b] = ld_u8_or(spv + gr, av != 0 && code, 127u);
            if (C::kNslab == 8 && b == 1) {
#pragma unroll
              for (int q = 0; q < 3; ++q) vp[q] = ld_or_zero(src + 16 * (q + 1), av != 0 && !code);
            }
          }
          row1 = row;
          sc1 = sc;
          pos2 = pos3 < L ? pos3 : -1;
          {
            const int pi = pos2 >> P.log2_ps;
            page2 = ld_i32_or(P.block_table + (int64_t)r * P.max_pages + pi, !runs && pos2 >= 0 && pi < P.max_pages,
                              runs ? pi : -1);
          }
          {
            const int kk = (lo + 2 * (t + 4) + my_half) * kBlockRows + w8 + (lane & 7);
            const bool in = kk < hi * kBlockRows && lane < 16;
            if (runs) {
              const int4 rn = reinterpret_cast<const int4*>(runs)[tok];
              pos3 = in && kk < rn.w ? (kk < rn.y ? rn.x + kk : rn.z + kk - rn.y) : -1;
            } else {
              pos3 = ld_i32_or(P.indices + (int64_t)tok * P.topk + kk, sparse && in && kk < P.topk,
                               sparse || !in ? -1 : kk);
            }
          }
        }
      });
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the even CTA's MMAs into both CTAs' TMEM have completed
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <int LAYOUT>
constexpr size_t kSmemBytes = Cfg<LAYOUT>::kOffMisc + sizeof(PairMisc) + 1024;

template <int LAYOUT>
cudaError_t launch(const DecodeParams& p, const CUtensorMap& q_map, int clusters, cudaStream_t stream) {
  auto kern = mla_decode_pair_fp4_kernel<LAYOUT>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes<LAYOUT>));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(2 * clusters), dim3(kPairThreads), kSmemBytes<LAYOUT>, stream, p, q_map);
}

template <int LAYOUT>
cudaError_t max_clusters(int* clusters) {
  auto kern = mla_decode_pair_fp4_kernel<LAYOUT>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes<LAYOUT>));
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms & ~1);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kSmemBytes<LAYOUT>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(clusters, kern, &cfg);
}

}  // namespace

cudaError_t launch_decode_pair_fp4(int layout, const DecodeParams& p, const CUtensorMap& q_map, int clusters,
                                   cudaStream_t stream) {
  return layout == 3 ? launch<3>(p, q_map, clusters, stream) : launch<4>(p, q_map, clusters, stream);
}

cudaError_t decode_pair_fp4_max_clusters(int layout, int* clusters) {
  return layout == 3 ? max_clusters<3>(clusters) : max_clusters<4>(clusters);
}

}  // namespace mla
