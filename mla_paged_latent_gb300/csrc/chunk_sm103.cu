// Attention of a chunk of new tokens over the paged latent cache, in the per-head ("compute friendly") form
// ("mla_attention.py · tduncan/Nvidia-Optimization-Stack-VLLM", module docstring, Compute Friendly Approach: k_nope and v
// of every head are produced from kv_c by the up-projection, k_pe is shared by the heads).
//
// With c_j the latent row and r_j the RoPE part of cached row j, head h attends with K_j = [W_k[h] c_j | r_j] (192) and
// V_j = W_v[h] c_j (128): 640 operations a (query, row, head) against 2176 of the absorbed form, for 2^18 operations a
// (row, head) once. Three steps on one stream, and a fourth where the rows are few:
//   chunk_rows_kernel  the requests' rows, in order, as bf16 [rows, 576]; each request starts at a multiple of 128 and the
//                      rows up to the next are zeros, so that a masked row is never what memory happened to hold;
//   the product of the latent part with W (gemm_pair_kernel), K and V of a group of heads rounded to bf16 [rows, heads, 256]
//                      (operands of the tensor cores; the sums are fp32), which attention then reads many times;
//   chunk_attention_kernel;
//   chunk_merge_kernel where a query tile was split over the rows.
#include <cstdint>
#include <cuda_runtime.h>

#include "decode_common.cuh"
#include "kv_row.cuh"
#include "mla_kernels.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

// ----------------------------------------------------------------------------- rows
// One warp a row. Bound by the bytes: the stored row in, 1152 bytes out.
template <int LAYOUT>
__global__ void __launch_bounds__(256) chunk_rows_kernel(const __grid_constant__ ChunkParams P) {
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= P.kv_rows) return;
  const int req = P.tile_req[row >> 7];
  const int4 r = reinterpret_cast<const int4*>(P.requests)[req];  // q_start, q_len, kv_start, kv_len
  const int pos = row - r.z;
  uint4* dst = reinterpret_cast<uint4*>(P.rows + static_cast<int64_t>(row) * 576);
  int page = -1;
  if (pos < r.w) {
    const int pi = pos >> P.log2_ps;
    if (pi < P.max_pages) page = P.block_table[static_cast<int64_t>(req) * P.max_pages + pi];
    if (page < 0 || page >= P.num_pages) {  // reported, read as zeros
      if (lane == 0) atomicOr(P.status, 2u);
      page = -1;
    }
  }
  if (page < 0) {
    dst[lane] = make_uint4(0, 0, 0, 0);
    dst[32 + lane] = make_uint4(0, 0, 0, 0);
    if (lane < 8) dst[64 + lane] = make_uint4(0, 0, 0, 0);
    return;
  }
  read_row<LAYOUT>(P.kv + page * P.page_bytes, pos & (P.page_size - 1), P.page_size, lane, dst);
}

// ----------------------------------------------------------------------------- attention
// A pair of SMs (one tensor-core pair) takes a unit: up to 512 query rows of one request and head against a range of
// KV tiles of 128 rows. The rows are two sub-tiles of 256, 128 in each CTA, so that one sub-tile's products run under the
// other's softmax:
//   S = Q K^T   M = 256, N = 128 (each CTA holds 64 of the tile's rows), K = 192: 12 instructions
//   O += P V    M = 256, N = 128 (each CTA holds 64 of the value dims), K = 128: 8 instructions, P from TMEM
// Single SMs would need all of K and V in each: 80 KB a tile instead of 40, more than shared memory brings in under the
// products, and only one tile and a half fit beside Q.
// TMEM: S of the two sub-tiles (128 columns each; P as bf16 pairs takes the first 64 once S has been read) and O (128 each).
// Products are issued in the order PV0(j) S0(j+1) PV1(j) S1(j+1): S(j+1) follows the PV(j) that reads P from the same
// columns, and its completion says that O holds tile j, so a rescale of O needs no barrier of its own.
// P is rounded to bf16, an operand of the tensor cores; maxima, sums and O are fp32. The running maximum moves (and O is
// rescaled) only when a tile exceeds it by 2^32, so a row's sum stays below rows x 2^32 x max |V|.
// Shared memory per CTA: Q 2 x 48 KB, and 3 stages of K (64 rows x 192) and V (128 rows x 64 dims), 40 KB each.
//   warp 0      TMA            warp 1      TMEM, MMA issue (even CTA)
//   warps 4-7   softmax and epilogue of sub-tile 0, warps 8-11 of sub-tile 1: a query row a thread
constexpr int kChunkThreads = 384;
constexpr uint32_t kQSlab = 128 * 128;
constexpr uint32_t kQSub = 3 * kQSlab;
constexpr uint32_t kKSlab = 64 * 128;
constexpr uint32_t kKBytes = 3 * kKSlab;
constexpr uint32_t kVBytes = 128 * 128;
constexpr int kKvStages = 3;
constexpr uint32_t kOffK = 2 * kQSub;
constexpr uint32_t kOffV = kOffK + kKvStages * kKBytes;
constexpr uint32_t kOffChunkMisc = kOffV + kKvStages * kVBytes;
constexpr float kChunkRescaleLog2 = 32.0f;

struct ChunkMisc {
  uint64_t q_full[2], q_empty[2];                  // full barriers and p_full, o_free: in the even CTA, both CTAs arrive
  uint64_t k_full[kKvStages], k_empty[kKvStages];  // the others: in each CTA, by multicast commits
  uint64_t v_full[kKvStages], v_empty[kKvStages];
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t last;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kChunkSmem = kOffChunkMisc + sizeof(ChunkMisc) + 1024;
static_assert(kChunkSmem <= 232448, "shared memory budget of one CTA");

struct Unit {
  int q_start, q0, n, kv_start, len, head, tb, slot;
  int tiles[2];  // KV tiles of each sub-tile, from tb on
};

// KV rows that query i of n sees: those before its limit.
__device__ __forceinline__ int row_limit(int causal, int len, int n, int i) {
  return causal ? min(len, len - n + i + 1) : len;
}

__device__ __forceinline__ Unit read_unit(const ChunkParams& P, int item) {
  const int4 a = reinterpret_cast<const int4*>(P.items)[2 * item];      // request, q0, head, first tile
  const int4 b = reinterpret_cast<const int4*>(P.items)[2 * item + 1];  // last tile + 1, slot or -1
  const int4 r = reinterpret_cast<const int4*>(P.requests)[a.x];
  Unit u;
  u.q_start = r.x;
  u.n = r.y;
  u.kv_start = r.z;
  u.len = r.w;
  u.q0 = a.y;
  u.head = a.z;
  u.tb = a.w;
  u.slot = b.y;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int last = min(u.q0 + 256 * (s + 1), u.n) - 1;
    const int lim = row_limit(P.causal, u.len, u.n, last);
    const int t = min(lim <= 0 ? 0 : (lim + 127) >> 7, b.x) - u.tb;
    u.tiles[s] = u.q0 + 256 * s >= u.n || u.head >= P.group_heads || t < 0 ? 0 : t;
  }
  return u;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kChunkThreads, 1)
    chunk_attention_kernel(const __grid_constant__ ChunkParams P, const __grid_constant__ CUtensorMap q_map,
                           const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap rope_map) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  ChunkMisc* misc = reinterpret_cast<ChunkMisc*>(smem + kOffChunkMisc);
  volatile int* abort_flag = &misc->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  auto here = [&](uint64_t& b) -> uint32_t { return smem_addr(&b); };
  auto lead = [&](uint64_t& b) -> uint32_t { return map_shared_rank(smem_addr(&b), 0); };
  auto wait = [&](uint64_t& b, uint32_t parity) -> bool { return wait_bar(smem_addr(&b), parity & 1, abort_flag, P.status); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(here(misc->q_full[s]), 2);
      mbar_init(here(misc->q_empty[s]), 1);
      mbar_init(here(misc->s_full[s]), 1);
      mbar_init(here(misc->p_full[s]), 8);
      mbar_init(here(misc->o_full[s]), 1);
      mbar_init(here(misc->o_free[s]), 8);
    }
    for (int s = 0; s < kKvStages; ++s) {
      mbar_init(here(misc->k_full[s]), 2);
      mbar_init(here(misc->k_empty[s]), 1);
      mbar_init(here(misc->v_full[s]), 2);
      mbar_init(here(misc->v_empty[s]), 1);
    }
    mbar_init(here(misc->last), 1);
    misc->abort = 0;
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
  const int pair = static_cast<int>(cluster_id_x());
  const int item0 = P.pair_items[pair], item1 = P.pair_items[pair + 1];

  if (warp < 4) {
    // 128 x 88 + 256 x 208 = the launch's 384 x 168 registers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0 && lane == 0) {
      tma_prefetch_desc(&q_map);
      tma_prefetch_desc(&kv_map);
      tma_prefetch_desc(&rope_map);
      int it = 0;            // KV tiles loaded
      int qn[2] = {0, 0};    // query sub-tiles loaded
      bool ok = true;
      for (int i = item0; i < item1 && ok; ++i) {
        const Unit u = read_unit(P, i);
        const int head = P.head0 + u.head;
        const int nt = max(u.tiles[0], u.tiles[1]);
        auto load_q = [&](int s) {
          if (u.tiles[s] == 0) return true;
          if (qn[s] > 0 && !wait(misc->q_empty[s], qn[s] - 1)) return false;
          const uint32_t full = lead(misc->q_full[s]);
          mbar_arrive_expect_tx_cluster(full, kQSub);
          for (int k = 0; k < 3; ++k)
            tma_load_3d_pair(sb + s * kQSub + k * kQSlab, &q_map, 64 * k, head, u.q_start + u.q0 + 256 * s + 128 * rank,
                             full);
          ++qn[s];
          return true;
        };
        auto load_k = [&](int j) {
          const int st = (it + j) % kKvStages, use = (it + j) / kKvStages;
          if (use > 0 && !wait(misc->k_empty[st], use - 1)) return false;
          const uint32_t full = lead(misc->k_full[st]), at = sb + kOffK + st * kKBytes;
          const int row = u.kv_start + (u.tb + j) * 128 + 64 * rank;
          mbar_arrive_expect_tx_cluster(full, kKBytes);
          tma_load_2d_pair(at, &kv_map, u.head * 256, row, full);
          tma_load_2d_pair(at + kKSlab, &kv_map, u.head * 256 + 64, row, full);
          tma_load_2d_pair(at + 2 * kKSlab, &rope_map, 512, row, full);
          return true;
        };
        auto load_v = [&](int j) {
          const int st = (it + j) % kKvStages, use = (it + j) / kKvStages;
          if (use > 0 && !wait(misc->v_empty[st], use - 1)) return false;
          const uint32_t full = lead(misc->v_full[st]), at = sb + kOffV + st * kVBytes;
          const int row = u.kv_start + (u.tb + j) * 128, dim = u.head * 256 + 128 + 64 * rank;
          mbar_arrive_expect_tx_cluster(full, kVBytes);
          tma_load_2d_pair(at, &kv_map, dim, row, full);
          tma_load_2d_pair(at + kVBytes / 2, &kv_map, dim, row + 64, full);
          return true;
        };
        ok = load_q(0);
        for (int j = 0; j < nt && ok; ++j) {
          ok = load_k(j);
          if (j == 0 && ok) ok = load_q(1);
          if (ok) ok = load_v(j);
        }
        it += nt;
      }
      if (*abort_flag && rank == 0) {
        // copies still in flight land on this CTA's barriers: wait for them (bounded)
        for (int s = 0; s < 2; ++s)
          if (qn[s] > 0) mbar_wait_drain_cluster(here(misc->q_full[s]), (qn[s] - 1) & 1);
        for (int st = 0; st < kKvStages; ++st) {
          mbar_wait_drain_cluster(here(misc->k_full[st]), 0);
          mbar_wait_drain_cluster(here(misc->k_full[st]), 1);
          mbar_wait_drain_cluster(here(misc->v_full[st]), 0);
          mbar_wait_drain_cluster(here(misc->v_full[st]), 1);
        }
      }
    } else if (warp == 1 && rank == 0 && lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(256, 128, 0, 0);
      constexpr uint32_t idesc_o = idesc_bf16_f32(256, 128, 0, 1);  // V: MN-major, 64 dims of each CTA
      const uint64_t kmaj = sdesc_sw128(0, 16, 1024);
      const uint64_t vmaj = sdesc_sw128(0, kVBytes, 1024);
      int it = 0;
      int units[2] = {0, 0}, scores[2] = {0, 0};  // per sub-tile: units begun, score tiles whose P has been waited for
      bool ok = true;
      for (int i = item0; i < item1 && ok; ++i) {
        const Unit u = read_unit(P, i);
        const int nt = max(u.tiles[0], u.tiles[1]);
        // the last of the sub-tiles that use tile j
        auto last_user = [&](int s, int j) { return s == 1 || j >= u.tiles[1]; };
        auto issue_s = [&](int s, int j) {
          const int st = (it + j) % kKvStages, use = (it + j) / kKvStages;
          if (!wait(misc->k_full[st], use)) return false;
          tc_fence_after();
          const uint64_t q = kmaj | ((sb + s * kQSub) >> 4);
          const uint64_t k = kmaj | ((sb + kOffK + st * kKBytes) >> 4);
#pragma unroll
          for (int x = 0; x < 12; ++x)
            mma_bf16_pair(tmem + s * 128, q + (x >> 2) * (kQSlab >> 4) + (x & 3) * 2,
                          k + (x >> 2) * (kKSlab >> 4) + (x & 3) * 2, idesc_s, x ? 1u : 0u);
          mma_commit_pair(here(misc->s_full[s]), 3);
          if (last_user(s, j)) mma_commit_pair(here(misc->k_empty[st]), 3);
          if (j + 1 == u.tiles[s]) mma_commit_pair(here(misc->q_empty[s]), 3);
          return true;
        };
        for (int s = 0; s < 2 && ok; ++s)
          if (u.tiles[s] > 0) ok = wait(misc->q_full[s], units[s]) && issue_s(s, 0);
        for (int j = 0; j < nt && ok; ++j) {
          const int st = (it + j) % kKvStages, use = (it + j) / kKvStages;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok || j >= u.tiles[s]) continue;
            ok = wait(misc->p_full[s], scores[s]);
            if (ok && j == 0 && units[s] > 0) ok = wait(misc->o_free[s], units[s] - 1);
            if (ok) ok = wait(misc->v_full[st], use);
            if (!ok) continue;
            ++scores[s];
            tc_fence_after();
            const uint64_t v = vmaj | ((sb + kOffV + st * kVBytes) >> 4);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              mma_bf16_pair_ts(tmem + 256 + s * 128, tmem + s * 128 + 8 * x, v + x * (2048 >> 4), idesc_o,
                               (j | x) ? 1u : 0u);
            if (last_user(s, j)) mma_commit_pair(here(misc->v_empty[st]), 3);
            if (j + 1 == u.tiles[s]) mma_commit_pair(here(misc->o_full[s]), 3);
            else ok = issue_s(s, j + 1);
          }
        }
        it += nt;
        for (int s = 0; s < 2; ++s) units[s] += u.tiles[s] > 0;
      }
      mma_commit_pair(here(misc->last), 1);
      mbar_wait_drain_cluster(here(misc->last), 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int s = (warp - 4) >> 2, quarter = warp & 3;
    const int mine = 256 * s + 128 * rank + 32 * quarter + lane;  // row of the unit
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_off + s * 128, t_o = tmem + lane_off + 256 + s * 128;
    const float2 scale2 = make_float2(P.scale_log2, P.scale_log2);
    int scores = 0, units = 0;
    bool ok = true;
    for (int i = item0; i < item1 && ok; ++i) {
      const Unit u = read_unit(P, i);
      if (u.head >= P.group_heads) continue;
      const int row = u.q0 + mine;  // query of the request
      const int lim = row_limit(P.causal, u.len, u.n, row);
      const int tiles = u.tiles[s];
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < tiles; ++j) {
        if (!wait(misc->s_full[s], scores)) {
          ok = false;
          break;
        }
        ++scores;
        tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32(t_s + 32 * k, x + 32 * k);
        tmem_wait_ld();
        const int nv = lim - (u.tb + j) * 128;  // columns that this row sees
        if (__any_sync(0xffffffffu, nv < 128)) {
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (k >= nv) x[k] = 0xFF800000u;
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 64; ++k)
          m4[k & 3] = max3(m4[k & 3], __uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
        const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * P.scale_log2;
        const bool raise = mt > m_run + kChunkRescaleLog2;
        if (__any_sync(0xffffffffu, raise)) {
          const float a = raise ? fast_exp2(m_run - mt) : 1.f;  // (0 for the first rows that a query sees)
          l_run *= a;
          if (raise) m_run = mt;
          if (j > 0) {
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              uint32_t o[32];
              tmem_ld32(t_o + 32 * k, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
              tmem_st32(t_o + 32 * k, o);
            }
          }
        }
        const float m_use = m_run == -INFINITY ? 0.f : m_run;
        const float2 neg = make_float2(-m_use, -m_use);
        float2 sum[2] = {make_float2(l_run, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float2 v = fma2(make_float2(__uint_as_float(x[64 * h + 2 * k]), __uint_as_float(x[64 * h + 2 * k + 1])),
                                  scale2.x, neg);
            const float2 e = make_float2(fast_exp2(v.x), fast_exp2(v.y));
            sum[k & 1] = add2(sum[k & 1], e);
            p[k] = f32x2_to_bf16x2(e.x, e.y);
          }
          tmem_st32(t_s + 32 * h, p);
        }
        const float2 t = add2(sum[0], sum[1]);
        l_run = t.x + t.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(misc->p_full[s]));
      }
      if (!ok) break;
      // Out, 32 bytes a store. A row that sees nothing is zeros with an lse of -infinity; a NaN sum stays NaN.
      const bool empty = l_run == 0.f;
      const float inv = empty ? 0.f : 1.0f / l_run;
      const float lse = empty ? -INFINITY : (m_run + log2f(l_run)) * 0.6931471805599453f;
      const bool live = row < u.n;
      if (tiles > 0) {
        if (!wait(misc->o_full[s], units)) break;
        ++units;
        tc_fence_after();
      }
      const int64_t at = static_cast<int64_t>(u.q_start + row) * P.heads + P.head0 + u.head;  // row of out
      const int64_t part = static_cast<int64_t>(u.slot) * 512 + mine;
      if (live) {
        if (u.slot >= 0) P.part_lse[part] = lse;
        else if (P.lse != nullptr) P.lse[at] = lse;
      }
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        uint32_t o[32];
        __syncwarp();
        if (tiles > 0) {
          tmem_ld32(t_o + 32 * k, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = empty ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);
        if (live && u.slot >= 0) {
          float* dst = P.part_out + part * 128 + 32 * k;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t v[8] = {o[8 * e], o[8 * e + 1], o[8 * e + 2], o[8 * e + 3],
                                   o[8 * e + 4], o[8 * e + 5], o[8 * e + 6], o[8 * e + 7]};
            st_global_v8(dst + 8 * e, v);
          }
        } else if (live) {
          uint16_t* dst = P.out + at * 128 + 32 * k;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t v[8];
#pragma unroll
            for (int y = 0; y < 8; ++y)
              v[y] = f32x2_to_bf16x2(__uint_as_float(o[16 * e + 2 * y]), __uint_as_float(o[16 * e + 2 * y + 1]));
            st_global_v8(dst + 16 * e, v);
          }
        }
      }
      if (tiles > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(misc->o_free[s]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the even CTA's MMAs into both CTAs' TMEM have completed
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ----------------------------------------------------------------------------- merge
// out = sum_p e^(lse_p - lse) out_p over the pieces of a query tile ("mla_attention.py ·
// tduncan/Nvidia-Optimization-Stack-VLLM", Chunked Prefill: merge_attn_states). One warp a row, four dims a lane; a piece
// that saw nothing has lse -infinity and weight 0, a NaN is passed on.
__global__ void __launch_bounds__(256) chunk_merge_kernel(const __grid_constant__ ChunkParams P) {
  pdl_trigger();
  pdl_wait();
  const int tile = blockIdx.x >> 6;
  const int mine = (blockIdx.x & 63) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int4 a = reinterpret_cast<const int4*>(P.merges)[2 * tile];      // request, q0, head, first slot
  const int4 b = reinterpret_cast<const int4*>(P.merges)[2 * tile + 1];  // pieces
  const int4 r = reinterpret_cast<const int4*>(P.requests)[a.x];
  if (a.z >= P.group_heads || a.y + mine >= r.y) return;
  float top = -INFINITY;
  bool any = false;
  for (int p = 0; p < b.x; ++p) {
    const float l = P.part_lse[static_cast<int64_t>(a.w + p) * 512 + mine];
    top = fmaxf(top, l);
    any |= l != -INFINITY;
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
  if (any)
    for (int p = 0; p < b.x; ++p) {
      const int64_t part = static_cast<int64_t>(a.w + p) * 512 + mine;
      const float l = P.part_lse[part];
      if (l == -INFINITY) continue;
      const float w = expf(l - top);
      const float4 v = reinterpret_cast<const float4*>(P.part_out + part * 128)[lane];
      total += w;
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  const float inv = any ? 1.0f / total : 0.f;
  const int64_t at = static_cast<int64_t>(r.x + a.y + mine) * P.heads + P.head0 + a.z;
  reinterpret_cast<uint2*>(P.out + at * 128)[lane] =
      make_uint2(f32x2_to_bf16x2(acc.x * inv, acc.y * inv), f32x2_to_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0 && P.lse != nullptr) P.lse[at] = any ? top + logf(total) : -INFINITY;
}

}  // namespace

cudaError_t launch_chunk_rows(int layout, const ChunkParams& p, cudaStream_t stream) {
  const dim3 grid((p.kv_rows + 7) / 8), block(256);
  switch (layout) {
    case 0: return launch_pdl(chunk_rows_kernel<0>, grid, block, 0, stream, p);
    case 2: return launch_pdl(chunk_rows_kernel<2>, grid, block, 0, stream, p);
    default: return launch_pdl(chunk_rows_kernel<4>, grid, block, 0, stream, p);
  }
}

cudaError_t launch_chunk_attention(const ChunkParams& p, const CUtensorMap& q_map, const CUtensorMap& kv_map,
                                   const CUtensorMap& rope_map, int pairs, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(chunk_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kChunkSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_attention_kernel, dim3(2 * pairs), dim3(kChunkThreads), kChunkSmem, stream, p, q_map, kv_map,
                    rope_map);
}

cudaError_t launch_chunk_merge(const ChunkParams& p, int merges, cudaStream_t stream) {
  return launch_pdl(chunk_merge_kernel, dim3(64 * merges), dim3(256), 0, stream, p);
}

}  // namespace mla
