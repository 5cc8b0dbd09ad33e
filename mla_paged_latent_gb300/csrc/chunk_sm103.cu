// Attention of a chunk of new tokens over the paged latent cache, in the per-head ("compute friendly") form
// ("mla_attention.py · tduncan/Nvidia-Optimization-Stack-VLLM", module docstring, Compute Friendly Approach: k_nope and v
// of every head are produced from kv_c by the up-projection, k_pe is shared by the heads).
//
// With c_j the latent row and r_j the RoPE part of cached row j, head h attends with K_j = [W_k[h] c_j | r_j] (192) and
// V_j = W_v[h] c_j (128): 640 operations a (query, row, head) against 2176 of the absorbed form, for 2^18 operations a
// (row, head) once. Three steps on one stream, and a fourth where the rows are few:
//   chunk_rows_kernel  the requests' rows, in order, as bf16 [rows, 576]; each request starts at a multiple of 128 and the
//                      rows up to the next are zeros, so that a masked row is never what memory happened to hold;
//   the product of the latent part with W (gemm_pair_kernel), K (bf16) and V (fp16 or bf16) of a group of heads
//                      [rows, heads, 256] (operands of the tensor cores; the sums are fp32), which attention then reads many times;
//   chunk_attention_kernel;
//   chunk_merge_kernel where a query tile was split over the rows.
// One after the other on 2048 queries after 32768 bf16 rows at 128 heads: 13, 742 and 3150 us (1.80 PFLOP/s of 640 operations a
// query, row and head; in a loop the power limit makes 4.3 to 4.4 ms of the three).
#include <cstdint>
#include <cuda_runtime.h>

#include "decode_common.cuh"
#include "kv_row.cuh"
#include "mla_kernels.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

// ----------------------------------------------------------------------------- rows
// One warp a row. Bound by the bytes: the stored row in, 1152 bytes out (65736 bf16 rows in 21 us, 7 TB/s in and out).
template <int LAYOUT>
__global__ void __launch_bounds__(256) chunk_rows_kernel(const __grid_constant__ ChunkParams P) {
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i * P.group_heads < P.heads; i += 256) P.any_wide[i] = 0;
  if (row >= P.kv_rows) return;
  const int4 tile = reinterpret_cast<const int4*>(P.kv_tiles)[row >> 7];  // request, position of the first row, kv_len
  const int req = tile.x, pos = tile.y + (row & 127);
  uint4* dst = reinterpret_cast<uint4*>(P.rows + static_cast<int64_t>(row) * 576);
  int page = -1;
  if (pos < tile.z) {
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
  const bool bad = read_row<LAYOUT>(P.kv + page * P.page_bytes, pos & (P.page_size - 1), P.page_size, lane, dst);
  // An infinity or NaN in the latent part would be one in all of V, and 0 times it NaN for queries of the tile that do not see the
  // row. It goes into the key instead, whose scores are masked: NaN for those that see it.
  if (__any_sync(0xffffffffu, bad)) {
    dst[lane] = make_uint4(0, 0, 0, 0);
    dst[32 + lane] = make_uint4(0, 0, 0, 0);
    if (lane < 8) dst[64 + lane] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
  }
}

// ----------------------------------------------------------------------------- attention
// A pair of SMs (one tensor-core pair) takes a unit: up to 512 query rows of one request and head against a range of
// KV tiles of 128 rows. The rows are two sub-tiles of 256, 128 in each CTA, so that one sub-tile's products run under the
// other's softmax:
//   S = Q K^T   M = 256, N = 128 (each CTA holds 64 of the tile's rows), K = 192: 12 instructions
//   O += P V    M = 256, N = 128 (each CTA holds 64 of the value dims), K = 128: 8 instructions, P from TMEM
// Single SMs would need all of K and V in each: 80 KB a tile instead of 40, more than shared memory brings in under the
// products, and only one tile and a half fit beside Q.
// TMEM: S of the two sub-tiles (128 columns each; P as fp16 pairs takes the first 64 once S has been read) and O (128 each).
// A thread for each sub-tile issues PV(j) S(j+1) in turn: S(j+1) follows the PV(j) that reads P from the same columns, and
// its completion says that O holds tile j, so a rescale of O needs no barrier of its own.
// Bound by the tensor cores in the end: 2 x 1280 cycles of products a KV tile and unit. One issuing thread took 4790 (its barrier
// tests and commits stood between the products), two that run freely 5040 (both softmaxes at once); turns 3730, stages passed on by
// the softmax warps 3560, P in halves and nothing spilled 3090 (traced again, at other clocks: 3250, with values in bf16 3430; one
// sub-tile alone 2880 and 3050).
// P and V are fp16 where the values of 32 rows are of a size that fp16 holds well, and bf16 where they are not (an instruction has
// 16 rows, so its type may differ from the next one's): a scale of V for every 32 rows, which P makes good, would cost the weights of
// rows whose values are smaller by far their bits. P is kept below 2^15 by a reference that moves (and O is rescaled) only
// when a tile exceeds it by 2^8. Both in bf16 are off by 0.0027 of the result against 0.0020 (in the mean square; the result's own
// rounding is 0.0017). Maxima, sums and O are fp32.
// Shared memory per CTA: Q 2 x 48 KB, and 3 stages of K (64 rows x 192) and V (128 rows x 64 dims), 40 KB each.
//   warp 0      TMA            warps 1, 2  MMA issue of sub-tile 0 and 1 (even CTA); warp 1 TMEM
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
constexpr float kWeightLog2 = 7.0f, kWeightMaxLog2 = 15.0f;

struct ChunkMisc {
  uint64_t q_full[2], q_empty[2];                  // full barriers and p_full, o_free: in the even CTA, both CTAs arrive
  uint64_t k_full[kKvStages], k_empty[kKvStages];  // the others: in each CTA (empty: its two sub-tiles arrive)
  uint64_t v_full[kKvStages], v_empty[kKvStages];
  uint64_t s_full[2], p_full[4], o_full[2], o_free[2];  // p_full: halves of the KV tile, of each sub-tile
  uint64_t turn[2];                                // of the two MMA threads
  uint64_t last;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kChunkSmem = kOffChunkMisc + sizeof(ChunkMisc) + 1024;
static_assert(kChunkSmem <= 232448, "shared memory budget of one CTA");

// High word of every descriptor here: 1024 bytes between groups of eight rows, version 1, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

struct Unit {
  int q_start, q0, n, kv_start, len, head, tb, slot;
  int tiles[2];  // KV tiles of each sub-tile, from tb on
};

// KV rows that query i of n sees: those before its limit.
__device__ __forceinline__ int row_limit(int causal, int len, int n, int i) {
  return causal ? min(len, len - n + i + 1) : len;
}

__device__ __forceinline__ Unit read_unit(const ChunkParams& P, int item) {
  const int4 r = reinterpret_cast<const int4*>(P.items)[3 * item];      // q_start, q_len, kv_start, kv_len
  const int4 a = reinterpret_cast<const int4*>(P.items)[3 * item + 1];  // q0, head, first tile, last tile + 1
  const int slot = P.items[12 * item + 8];                              // or -1
  Unit u;
  u.q_start = r.x;
  u.n = r.y;
  u.kv_start = r.z;
  u.len = r.w;
  u.q0 = a.x;
  u.head = a.y;
  u.tb = a.z;
  u.slot = slot;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int last = min(u.q0 + 256 * (s + 1), u.n) - 1;
    const int lim = row_limit(P.causal, u.len, u.n, last);
    const int t = min(lim <= 0 ? 0 : (lim + 127) >> 7, a.w) - u.tb;
    u.tiles[s] = u.q0 + 256 * s >= u.n || u.head >= P.group_heads || t < 0 ? 0 : t;
  }
  return u;
}

// Of each KV tile of a unit: four bytes, one for 32 rows, 1 where their values (and so their weights) are bf16.
__device__ __forceinline__ const uint32_t* wide_groups(const ChunkParams& P, const Unit& u) {
  return reinterpret_cast<const uint32_t*>(P.value_wide) + static_cast<int64_t>(u.head) * (P.kv_rows >> 7) + (u.kv_start >> 7) + u.tb;
}

// What the warps share.
struct ChunkCta {
  const ChunkParams& P;
  ChunkMisc* misc;
  uint32_t sb, tmem;   // shared memory, TMEM
  int item0, item1;    // this pair's units
  __device__ __forceinline__ uint32_t here(uint64_t& b) const { return smem_addr(&b); }
  __device__ __forceinline__ uint32_t lead(uint64_t& b) const { return map_shared_rank(smem_addr(&b), 0); }
  __device__ __forceinline__ bool wait(uint64_t& b, uint32_t parity) const {
    return wait_bar(smem_addr(&b), parity & 1, &misc->abort, P.status);
  }
};

// Warp 0, one thread: copies of Q, K and V.
__device__ __forceinline__ void chunk_load(const ChunkCta& C, const CUtensorMap& q_map, const CUtensorMap& kv_map,
                                           const CUtensorMap& rope_map) {
  const ChunkParams& P = C.P;
  ChunkMisc* misc = C.misc;
  const int rank = static_cast<int>(cluster_ctarank());
  int it = 0;            // KV tiles loaded
  int qn[2] = {0, 0};    // query sub-tiles loaded
  bool ok = true;
  for (int i = C.item0; i < C.item1 && ok; ++i) {
    const Unit u = read_unit(P, i);
    const int head = P.head0 + u.head;
    const int nt = max(u.tiles[0], u.tiles[1]);
    auto load_q = [&](int s) {
      if (u.tiles[s] == 0) return true;
      if (qn[s] > 0 && !C.wait(misc->q_empty[s], qn[s] - 1)) return false;
      const uint32_t full = C.lead(misc->q_full[s]);
      mbar_arrive_expect_tx_cluster(full, kQSub);
      for (int k = 0; k < 3; ++k)
        tma_load_3d_pair(C.sb + s * kQSub + k * kQSlab, &q_map, 64 * k, head, u.q_start + u.q0 + 256 * s + 128 * rank,
                         full);
      ++qn[s];
      return true;
    };
    auto load_k = [&](int j) {
      const int st = (it + j) % kKvStages, use = (it + j) / kKvStages;
      if (use > 0 && !C.wait(misc->k_empty[st], use - 1)) return false;
      const uint32_t full = C.lead(misc->k_full[st]), at = C.sb + kOffK + st * kKBytes;
      const int row = u.kv_start + (u.tb + j) * 128 + 64 * rank;
      mbar_arrive_expect_tx_cluster(full, kKBytes);
      tma_load_2d_pair(at, &kv_map, u.head * 256, row, full);
      tma_load_2d_pair(at + kKSlab, &kv_map, u.head * 256 + 64, row, full);
      tma_load_2d_pair(at + 2 * kKSlab, &rope_map, 512, row, full);
      return true;
    };
    auto load_v = [&](int j) {
      const int st = (it + j) % kKvStages, use = (it + j) / kKvStages;
      if (use > 0 && !C.wait(misc->v_empty[st], use - 1)) return false;
      const uint32_t full = C.lead(misc->v_full[st]), at = C.sb + kOffV + st * kVBytes;
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
  if (*static_cast<volatile int*>(&misc->abort) != 0 && rank == 0) {
    // copies still in flight land on this CTA's barriers: wait for them (bounded)
    for (int s = 0; s < 2; ++s)
      if (qn[s] > 0) mbar_wait_drain_cluster(C.here(misc->q_full[s]), (qn[s] - 1) & 1);
    for (int st = 0; st < kKvStages; ++st) {
      mbar_wait_drain_cluster(C.here(misc->k_full[st]), 0);
      mbar_wait_drain_cluster(C.here(misc->k_full[st]), 1);
      mbar_wait_drain_cluster(C.here(misc->v_full[st]), 0);
      mbar_wait_drain_cluster(C.here(misc->v_full[st]), 1);
    }
  }
}

// MIXED: values of some heads and rows are bf16, and so are their weights. Where none are, the types are constants: chosen at every
// instruction and conversion they cost a whole prompt's attention 4 % (1627 us against 1690), a lone sub-tile 1 %; chosen by a
// branch a tile still more.
//
// One thread a sub-tile s of the even CTA: the products.
// The two threads take turns, a tile each: sub-tiles that begin a tile at once would also need their P at once, and the
// tensor cores would wait for both softmaxes.
template <int s, bool MIXED>
__device__ __forceinline__ void chunk_issue(const ChunkCta& C) {
  const ChunkParams& P = C.P;
  ChunkMisc* misc = C.misc;
  constexpr uint32_t idesc_s = idesc_bf16_f32(256, 128, 0, 0);
  constexpr uint32_t idesc_o = idesc_f16_f32(256, 128, 0, 1);  // V: MN-major, 64 dims of each CTA
  constexpr uint32_t idesc_wide = idesc_bf16_f32(256, 128, 0, 1);
  // low words of the descriptors: start address, and a leading offset that neither layout uses
  const uint32_t q = ((C.sb + s * kQSub) >> 4) | (1u << 16), k0 = ((C.sb + kOffK) >> 4) | (1u << 16),
                 v0 = ((C.sb + kOffV) >> 4) | (1u << 16);
  const uint32_t t_s = C.tmem + s * 128, t_o = C.tmem + 256 + s * 128;
  int it = 0, units = 0, scores = 0, turns = 0;  // KV tiles, units begun, score tiles whose P has been waited for, turns taken
  bool ok = true;
  for (int i = C.item0; i < C.item1 && ok; ++i) {
    const Unit u = read_unit(P, i);
    const int nt = max(u.tiles[0], u.tiles[1]), tiles = u.tiles[s];
    auto issue_s = [&](int j) {  // K of tile j has landed
      const uint32_t k = k0 + (it + j) % kKvStages * (kKBytes >> 4);
#pragma unroll
      for (int x = 0; x < 12; ++x) {
        mma_bf16_pair_lo(t_s, q + (x >> 2) * (kQSlab >> 4) + (x & 3) * 2, kDescHi,
                         k + (x >> 2) * (kKSlab >> 4) + (x & 3) * 2, kDescHi, idesc_s, x ? 1u : 0u);
        // (the other thread sees its turn about when the rest has been issued)
        if (x == 8 && j > 0) mbar_arrive(C.here(misc->turn[1 - s]));
      }
      mma_commit_pair(C.here(misc->s_full[s]), 3);
      if (j + 1 == tiles) mma_commit_pair(C.here(misc->q_empty[s]), 3);
    };
    auto k_landed = [&](int j) { return C.wait(misc->k_full[(it + j) % kKvStages], (it + j) / kKvStages); };
    const uint32_t* wides = wide_groups(P, u);
    uint32_t wide_next = 0;
    if (tiles > 0) {
      if (MIXED) wide_next = wides[0];
      ok = C.wait(misc->q_full[s], units) && k_landed(0);
      if (!ok) break;
      tc_fence_after();
      issue_s(0);
    }
    for (int j = 0; j < nt; ++j) {
      const int st = (it + j) % kKvStages, use = (it + j) / kKvStages;
      if (j >= tiles) {  // the other sub-tile's alone
        if (!(ok = C.wait(misc->turn[s], s == 0 ? turns - 1 : turns))) break;
        ++turns;
        mbar_arrive(C.here(misc->turn[1 - s]));
        continue;
      }
      // Everything but P first: a thread that tests a barrier waits until the instructions that it has queued are
      // dispatched, and a commit costs as much as one or two of them, so neither stands between P's arrival, PV and
      // the next S (the softmax warps pass on the stages, which their own barriers say have been read).
      ok = C.wait(misc->v_full[st], use);
      if (ok && j + 1 < tiles) ok = k_landed(j + 1);
      if (ok && j == 0 && units > 0) ok = C.wait(misc->o_free[s], units - 1);
      uint32_t idesc[4];  // of 32 rows each
#pragma unroll
      for (int g = 0; g < 4; ++g) idesc[g] = MIXED && (wide_next >> (8 * g) & 1) ? idesc_wide : idesc_o;
      if (ok) ok = C.wait(misc->p_full[2 * s], scores);
      if (ok) ok = C.wait(misc->turn[s], s == 0 ? turns - 1 : turns);
      if (!ok) break;
      ++turns;
      tc_fence_after();
      const uint32_t v = v0 + st * (kVBytes >> 4);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        mma_bf16_pair_ts_lo(t_o, t_s + 8 * x, v + x * (2048 >> 4), kDescHi, idesc[x >> 1], (j | x) ? 1u : 0u);
      if (!(ok = C.wait(misc->p_full[2 * s + 1], scores))) break;
      tc_fence_after();
#pragma unroll
      for (int x = 4; x < 8; ++x)
        mma_bf16_pair_ts_lo(t_o, t_s + 8 * x, v + x * (2048 >> 4), kDescHi, idesc[x >> 1], 1u);
      if (MIXED && j + 1 < tiles) wide_next = wides[j + 1];
      ++scores;
      if (j + 1 < tiles) {
        issue_s(j + 1);
      } else {
        mma_commit_pair(C.here(misc->o_full[s]), 3);
        mbar_arrive(C.here(misc->turn[1 - s]));
      }
    }
    it += nt;
    units += tiles > 0;
  }
  mma_commit_pair(C.here(misc->last), 1);
  mbar_wait_drain_cluster(C.here(misc->last), 0);
}

// Warps 4 to 11: softmax and epilogue, a query row a thread.
template <bool MIXED>
__device__ __forceinline__ void chunk_softmax(const ChunkCta& C) {
  const ChunkParams& P = C.P;
  ChunkMisc* misc = C.misc;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int s = (warp - 4) >> 2, quarter = warp & 3;
  const int mine = 256 * s + 128 * rank + 32 * quarter + lane;  // row of the unit
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t t_s = C.tmem + lane_off + s * 128, t_o = C.tmem + lane_off + 256 + s * 128;
  const uint32_t p_bar[2] = {C.lead(misc->p_full[2 * s]), C.lead(misc->p_full[2 * s + 1])};
  int scores = 0, units = 0, it = 0;
  bool ok = true;
  for (int i = C.item0; i < C.item1 && ok; ++i) {
    const Unit u = read_unit(P, i);
    if (u.head >= P.group_heads) continue;
    const int tiles = u.tiles[s], others = u.tiles[1 - s];
    const int lim = row_limit(P.causal, u.len, u.n, u.q0 + mine) - u.tb * 128;  // rows that this query sees, from tb on
    // The stage of K or V of tile j has been read by this sub-tile's products, and by the other's if it has none there:
    // each of two arrivals says so for one of them.
    auto pass_on = [&](uint64_t (&empty)[kKvStages], int j) {
      if (quarter == 0 && lane == 0) {
        const uint32_t b = C.here(empty[(it + j) % kKvStages]);
        mbar_arrive(b);
        if (j >= others) mbar_arrive(b);
      }
      __syncwarp();
    };
    // Weights are 2^(score - ref) with ref such that they stay below 2^15.
    float ref = -INFINITY, l_run = 0.f;
    const uint32_t* wides = wide_groups(P, u);
    uint32_t wide_next = 0;
    if (MIXED && tiles > 0) wide_next = wides[0];
    for (int j = 0; j < tiles; ++j) {
      const uint32_t wide = wide_next;
      if (!C.wait(misc->s_full[s], scores)) {
        ok = false;
        break;
      }
      ++scores;
      tc_fence_after();
      uint32_t x[128];
#pragma unroll
      for (int k = 0; k < 4; ++k) tmem_ld32(t_s + 32 * k, x + 32 * k);
      tmem_wait_ld();
      if (MIXED && j + 1 < tiles) wide_next = wides[j + 1];  // (not before: the wait would be for this load too)
      const int nv = lim - j * 128;  // columns that this row sees
      if (__any_sync(0xffffffffu, nv < 128)) {
#pragma unroll
        for (int k = 0; k < 128; ++k)
          if (k >= nv) x[k] = 0xFF800000u;
      }
      float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < 64; ++k)
        tops[k & 3] = max3(tops[k & 3], __uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
      const float top = P.scale_log2 * fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
      const bool raise = top > ref + kWeightMaxLog2;
      if (__any_sync(0xffffffffu, raise)) {
        const float a = raise ? fast_exp2(ref - (top - kWeightLog2)) : 1.f;  // (0 for the first rows that a query sees)
        l_run *= a;
        if (raise) ref = top - kWeightLog2;
        if (j > 0) {
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {  // (16 columns: the scores fill the registers)
            uint32_t o[16];
            tmem_ld16(t_o + 16 * k, o);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * a);
            tmem_st16(t_o + 16 * k, o);
          }
        }
      }
      const float ref_use = ref == -INFINITY ? 0.f : ref;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const int g = 2 * h + gg;
          uint32_t p[16];
          const float2 off2 = make_float2(-ref_use, -ref_use);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 v = fma2(make_float2(__uint_as_float(x[32 * g + 2 * k]), __uint_as_float(x[32 * g + 2 * k + 1])),
                                  P.scale_log2, off2);
            const float2 w = make_float2(fast_exp2(v.x), fast_exp2(v.y));
            sum[k & 1] = add2(sum[k & 1], w);
            p[k] = MIXED && (wide >> (8 * g) & 1) ? f32x2_to_bf16x2(w.x, w.y) : f32x2_to_f16x2(w.x, w.y);
          }
          const float2 t = add2(sum[0], sum[1]);
          l_run += t.x + t.y;
          tmem_st16(t_s + 16 * g, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_bar[h]);
        __syncwarp();
      }
      pass_on(misc->k_empty, j);  // (only now: P is waited for, the stages have two tiles' time)
      if (j > 0) pass_on(misc->v_empty, j - 1);
    }
    if (!ok) break;
    // Out, 32 bytes a store. A row that sees nothing is zeros with an lse of -infinity; a NaN sum stays NaN.
    const bool empty = l_run == 0.f;
    const float inv = empty ? 0.f : 1.0f / (l_run * (1 << kValueLog2));
    const float lse = empty ? -INFINITY : (ref + log2f(l_run)) * 0.6931471805599453f;
    const Unit w = read_unit(P, i);  // (again: no register holds it while the scores fill them)
    const int row = w.q0 + mine;
    const bool live = row < w.n && w.q_start + row < P.tokens;  // (whatever a schedule says)
    if (tiles > 0) {
      if (!C.wait(misc->o_full[s], units)) break;
      ++units;
      pass_on(misc->v_empty, tiles - 1);
      tc_fence_after();
    }
    const int64_t at = static_cast<int64_t>(w.q_start + row) * P.heads + P.head0 + w.head;  // row of out
    const int64_t part = static_cast<int64_t>(w.slot) + mine;
    if (live) {
      if (w.slot >= 0) P.part_lse[part] = lse;
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
      if (live && w.slot >= 0) {
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
      if (lane == 0) mbar_arrive_cluster(C.lead(misc->o_free[s]));
    }
    it += max(w.tiles[0], w.tiles[1]);
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kChunkThreads, 1)
    chunk_attention_kernel(const __grid_constant__ ChunkParams P, const __grid_constant__ CUtensorMap q_map,
                           const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap rope_map) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  ChunkMisc* misc = reinterpret_cast<ChunkMisc*>(smem + kOffChunkMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  auto here = [&](uint64_t& b) -> uint32_t { return smem_addr(&b); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(here(misc->q_full[s]), 2);
      mbar_init(here(misc->q_empty[s]), 1);
      mbar_init(here(misc->s_full[s]), 1);
      mbar_init(here(misc->p_full[2 * s]), 8);
      mbar_init(here(misc->p_full[2 * s + 1]), 8);
      mbar_init(here(misc->o_full[s]), 1);
      mbar_init(here(misc->o_free[s]), 8);
      mbar_init(here(misc->turn[s]), 1);
    }
    for (int s = 0; s < kKvStages; ++s) {
      mbar_init(here(misc->k_full[s]), 2);
      mbar_init(here(misc->k_empty[s]), 2);
      mbar_init(here(misc->v_full[s]), 2);
      mbar_init(here(misc->v_empty[s]), 2);
    }
    mbar_init(here(misc->last), 2);
    misc->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&q_map);
    tma_prefetch_desc(&kv_map);
    tma_prefetch_desc(&rope_map);
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
  const ChunkCta C = {P, misc, sb, tmem, P.pair_items[pair], P.pair_items[pair + 1]};
  const bool mixed = *P.any_wide != 0;
  if (warp < 4) {
    // 128 x 72 + 256 x 216 = the launch's 384 x 168 registers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0 && lane == 0) {
      chunk_load(C, q_map, kv_map, rope_map);
    } else if (warp < 3 && rank == 0 && lane == 0) {
      if (!mixed) {
        if (warp == 1) chunk_issue<0, false>(C);
        else chunk_issue<1, false>(C);
      } else {
        if (warp == 1) chunk_issue<0, true>(C);
        else chunk_issue<1, true>(C);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    if (!mixed) chunk_softmax<false>(C);
    else chunk_softmax<true>(C);
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
  const int4 a = reinterpret_cast<const int4*>(P.merges)[2 * tile];      // first token, tokens, head, first slot
  const int4 b = reinterpret_cast<const int4*>(P.merges)[2 * tile + 1];  // pieces
  const int rows = a.y;
  if (a.z >= P.group_heads || mine >= rows || a.x + mine >= P.tokens) return;
  const float* lses = P.part_lse + a.w + mine;  // of piece p: p * rows further
  float top = -INFINITY;
  bool any = false;
  for (int p = lane; p < b.x; p += 32) {
    const float l = lses[static_cast<int64_t>(p) * rows];
    top = fmaxf(top, l);
    any |= l != -INFINITY;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  any = __any_sync(0xffffffffu, any);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
  if (any)
    for (int p0 = 0; p0 < b.x; p0 += 32) {
      const float l = p0 + lane < b.x ? lses[static_cast<int64_t>(p0 + lane) * rows] : -INFINITY;
      const float mine_w = l == -INFINITY ? 0.f : expf(l - top);
      const int n = min(32, b.x - p0);
      const float4* src = reinterpret_cast<const float4*>(P.part_out) + (a.w + static_cast<int64_t>(p0) * rows + mine) * 32 + lane;
#pragma unroll 4
      for (int p = 0; p < n; ++p) {
        const float w = __shfl_sync(0xffffffffu, mine_w, p);
        const float4 v = src[static_cast<int64_t>(p) * rows * 32];
        total += w;
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
      }
    }
  const float inv = any ? 1.0f / total : 0.f;
  const int64_t at = static_cast<int64_t>(a.x + mine) * P.heads + P.head0 + a.z;
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
