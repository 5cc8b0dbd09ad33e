// Queries and KV rows rotated by positions of several axes (time, height and width of images and video): the step before
// a decode or a chunk's attention, as qkv_norm_rope_kernel, where RoPE pair i of token t turns by the angle of
// positions[axis(i)][t] instead of one position's. One axis for all 32 pairs is the ordinary rotation.
#include <cstdint>
#include <cuda_runtime.h>

#include "kv_row.cuh"
#include "mla_kernels.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

constexpr int kAxesWarps = 8;

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  const uint32_t h[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = bf16_to_f32(h[k] & 0xFFFFu);
    v[2 * k + 1] = __uint_as_float(h[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                    f32x2_to_bf16x2(v[6], v[7]));
}

// Where a token's pairs take their angles: lane i holds the position of pair i's axis.
struct Places {
  int pos;
  bool ok, below;  // all of them inside the table; all negative (padding, with a negative slot)
  __device__ __forceinline__ Places(const AxesParams& P, int t, int lane) {
    const int axis = static_cast<int>(P.axis_of_pair >> (2 * lane)) & 3;
    pos = P.qkv.positions[static_cast<int64_t>(axis) * P.qkv.tokens + t];
    ok = __all_sync(0xffffffffu, pos >= 0 && pos < P.qkv.max_pos);
    below = __all_sync(0xffffffffu, pos < 0);
  }
};
__device__ __forceinline__ float2 angle_at(const float* freqs, int pos, int pair) {
  return reinterpret_cast<const float2*>(freqs)[static_cast<int64_t>(pos) * 32 + pair];
}

__device__ __forceinline__ uint32_t rotate2(uint32_t two, float2 cs) {
  const float x0 = __uint_as_float(two << 16), x1 = __uint_as_float(two & 0xFFFF0000u);
  return f32x2_to_bf16x2(x0 * cs.x - x1 * cs.y, x0 * cs.y + x1 * cs.x);
}

// The first blocks take the KV rows, one warp each, with the arithmetic of the other fused writes. The others take the
// queries: a warp has four heads of a token (192-wide rows) or one (the others). Bound by the bytes and, for those, by the
// loads in flight: full occupancy, and a warp asks for its rows before it looks at the positions.
// NOPE: the queries' NoPE part is read and written, for it is not q_out's own or is normalised.
template <int WIDTH, bool NOPE>
__global__ void __launch_bounds__(kAxesWarps * 32, 8) axes_kernel(const __grid_constant__ AxesParams A) {
  pdl_trigger();
  pdl_wait();
  const QkvParams& P = A.qkv;
  __shared__ __align__(16) uint16_t srow[kAxesWarps][576];
  const int wi = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) < P.kv_blocks) {
    const int t = blockIdx.x * kAxesWarps + wi;
    if (t >= P.tokens) return;
    const int slot = P.slots[t];
    if (slot < 0) return;
    const int page = slot >> (31 - __clz(P.page_size));  // (a power of two)
    const Places at(A, t, lane);
    const uint32_t bad = (page >= P.num_pages ? 4u : 0u) | (at.ok ? 0u : 8u);
    if (bad != 0u) {  // reported, not written
      if (lane == 0 && P.status != nullptr) atomicOr(P.status, bad);
      return;
    }
    const uint16_t* raw = P.kv_raw + (int64_t)t * P.kv_row_stride;
    if (WIDTH == 512) {
      int pos[8];  // of the pairs that lanes 28-31 turn
#pragma unroll
      for (int k = 0; k < 8; ++k) pos[k] = __shfl_sync(0xffffffffu, at.pos, 8 * (lane & 3) + k);
      norm_rope_row_by(raw, P.kv_weight, P.kv_eps, [&](int i, int k) { return angle_at(P.freqs, pos[k], i); }, 512, lane, srow[wi]);
    } else {
      norm_rope_row_by(raw, P.kv_weight, P.kv_eps, [&](int i, int) { return angle_at(P.freqs, at.pos, i); }, 576, lane, srow[wi]);
    }
    write_any_row(srow[wi], lane, P.kv, P.layout, page, slot & (P.page_size - 1), P.page_size, P.page_bytes);
    return;
  }
  constexpr int kHeads = WIDTH == 192 ? 4 : 1;
  // (the entry point keeps tokens * heads below 2^31)
  const uint32_t groups = (P.heads + kHeads - 1) / kHeads;
  const uint32_t w = (blockIdx.x - P.kv_blocks) * kAxesWarps + wi;
  const int t = static_cast<int>(w / groups);
  if (t >= P.tokens) return;
  const int n0 = static_cast<int>(w - t * groups) * kHeads;
  const uint16_t* qn = P.q_nope + t * P.nope_token_stride + n0 * P.nope_head_stride;
  const uint16_t* qp = P.q_pe + t * P.pe_token_stride + n0 * P.pe_head_stride;
  uint16_t* q = P.q_out + (static_cast<int64_t>(t) * P.heads + n0) * WIDTH;
  auto report = [&](const Places& at) {  // rows left as they were; reported unless they are padding
    if (lane == 0 && P.status != nullptr && !(at.below && P.slots[t] < 0)) atomicOr(P.status, 8u);
  };

  if (WIDTH == 192) {
    // 4 x 16 chunks of 16 bytes of the NoPE parts, two a lane, and 4 x 8 of the RoPE parts
    const int left = P.heads - n0, h = lane >> 4, hp = lane >> 3, c = lane & 7;
    uint4 u0, u1, up;
    if (NOPE) {
      if (h < left) u0 = reinterpret_cast<const uint4*>(qn + h * P.nope_head_stride)[lane & 15];
      if (h + 2 < left) u1 = reinterpret_cast<const uint4*>(qn + (h + 2) * P.nope_head_stride)[lane & 15];
    }
    if (hp < left) up = reinterpret_cast<const uint4*>(qp + hp * P.pe_head_stride)[c];
    const Places at(A, t, lane);
    if (!at.ok) return report(at);
    float2 cs[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) cs[k] = angle_at(P.freqs, __shfl_sync(0xffffffffu, at.pos, 4 * c + k), 4 * c + k);
    if (NOPE) {
      if (h < left) reinterpret_cast<uint4*>(q + h * WIDTH)[lane & 15] = u0;
      if (h + 2 < left) reinterpret_cast<uint4*>(q + (h + 2) * WIDTH)[lane & 15] = u1;
    }
    if (hp < left)
      reinterpret_cast<uint4*>(q + hp * WIDTH + 128)[c] =
          make_uint4(rotate2(up.x, cs[0]), rotate2(up.y, cs[1]), rotate2(up.z, cs[2]), rotate2(up.w, cs[3]));
    return;
  }

  // 64 chunks of 16 bytes, two a lane, normalised over their 512 elements where asked; the 576-wide rows' RoPE part is
  // a pair a lane, that of the 512-wide rows the last eight chunks
  const bool pe_lane = WIDTH == 512 && lane >= 24;
  uint4 u0, u1 = make_uint4(0, 0, 0, 0);
  uint32_t two = 0;
  if (NOPE) u0 = *reinterpret_cast<const uint4*>(qn + 8 * lane);
  if (NOPE || pe_lane) u1 = *reinterpret_cast<const uint4*>(pe_lane ? qp + 8 * (lane - 24) : qn + 256 + 8 * lane);
  if (WIDTH == 576) two = reinterpret_cast<const uint32_t*>(qp)[lane];
  const Places at(A, t, lane);
  if (!at.ok) return report(at);
  if (WIDTH == 512 || NOPE) {
    if (WIDTH == 512 || P.q_norm) {  // (a bf16 number goes through fp32 unchanged)
      float rinv = 1.f;
      float a[8];
      if (NOPE && P.q_norm) {
        float ss = 0.f, b[8];
        unpack8(u0, a);
        unpack8(u1, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(a[k], a[k], fmaf(b[k], b[k], ss));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rinv = 1.0f / sqrtf(ss * (1.0f / 512.0f) + P.q_eps);
      }
      // one chunk after the other: both at once would not fit the registers of full occupancy
      auto scaled = [&](uint4 u, int chunk) {
        unpack8(u, a);
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] *= rinv;
        if (P.q_weight != nullptr) {
          float g[8];
          unpack8(reinterpret_cast<const uint4*>(P.q_weight)[chunk], g);
#pragma unroll
          for (int k = 0; k < 8; ++k) a[k] *= g[k];
        }
      };
      if (NOPE && P.q_norm) {
        scaled(u0, lane);
        u0 = pack8(a);
        scaled(u1, 32 + lane);
      } else {
        unpack8(u1, a);
      }
      if (WIDTH == 512) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = 4 * (lane & 7) + k;
          const int pos = __shfl_sync(0xffffffffu, at.pos, i);
          if (pe_lane) {
            const float2 cs = angle_at(P.freqs, pos, i);
            const float x0 = a[2 * k], x1 = a[2 * k + 1];
            a[2 * k] = x0 * cs.x - x1 * cs.y;
            a[2 * k + 1] = x0 * cs.y + x1 * cs.x;
          }
        }
      }
      u1 = pack8(a);
    }
    if (NOPE) reinterpret_cast<uint4*>(q)[lane] = u0;
    if (NOPE || pe_lane) reinterpret_cast<uint4*>(q)[32 + lane] = u1;
  }
  if (WIDTH == 576) reinterpret_cast<uint32_t*>(q + 512)[lane] = rotate2(two, angle_at(P.freqs, at.pos, lane));
}

}  // namespace

cudaError_t launch_qkv_norm_rope_axes(const AxesParams& p, cudaStream_t stream) {
  AxesParams a = p;
  a.qkv.kv_blocks = (p.qkv.tokens + kAxesWarps - 1) / kAxesWarps;
  const int per = p.q_width == 192 ? 4 : 1;
  const int64_t warps = static_cast<int64_t>(p.qkv.tokens) * ((p.qkv.heads + per - 1) / per);
  const dim3 grid(static_cast<unsigned>(a.qkv.kv_blocks + (warps + kAxesWarps - 1) / kAxesWarps)), block(kAxesWarps * 32);
  auto go = [&](auto kern) { return launch_pdl(kern, grid, block, 0, stream, a); };
  if (p.q_width == 192) return go(p.copy_nope ? axes_kernel<192, true> : axes_kernel<192, false>);
  if (p.q_width == 576) return go(p.copy_nope ? axes_kernel<576, true> : axes_kernel<576, false>);
  return go(p.copy_nope ? axes_kernel<512, true> : axes_kernel<512, false>);
}

}  // namespace mla
