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

// The token's rows of the (cos, sin) table, one an axis. ok: every axis in use has a position inside the table; below: all
// of them are negative (padding, with a negative slot).
struct Angles {
  const float* row[4];
  uint64_t axis_of_pair;
  bool ok, below;
  __device__ __forceinline__ Angles(const AxesParams& P, int t) : axis_of_pair(P.axis_of_pair), ok(true), below(true) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      row[a] = P.qkv.freqs;
      if (!((P.used_axes >> a) & 1u)) continue;
      const int pos = P.qkv.positions[static_cast<int64_t>(a) * P.qkv.tokens + t];
      ok &= pos >= 0 && pos < P.qkv.max_pos;
      below &= pos < 0;
      row[a] = P.qkv.freqs + static_cast<int64_t>(pos) * 64;
    }
  }
  __device__ __forceinline__ float2 operator()(int i) const {
    const uint32_t a = static_cast<uint32_t>(axis_of_pair >> (2 * i)) & 3u;
    const float* f = a < 2u ? (a == 0u ? row[0] : row[1]) : (a == 2u ? row[2] : row[3]);
    return reinterpret_cast<const float2*>(f)[i];
  }
};

__device__ __forceinline__ uint32_t rotate2(uint32_t two, float2 cs) {
  const float x0 = __uint_as_float(two << 16), x1 = __uint_as_float(two & 0xFFFF0000u);
  return f32x2_to_bf16x2(x0 * cs.x - x1 * cs.y, x0 * cs.y + x1 * cs.x);
}

// The first blocks take the KV rows, one warp each, with the arithmetic of the other fused writes. The others take the
// queries: a warp holds its token's angles in registers (they are the same for all heads) and goes through `per` heads.
// Bound by the bytes and, for those, by the loads in flight.
template <int WIDTH>
__global__ void __launch_bounds__(kAxesWarps * 32) axes_kernel(const __grid_constant__ AxesParams A, int per) {
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
    const Angles angle(A, t);
    const uint32_t bad = (page >= P.num_pages ? 4u : 0u) | (angle.ok ? 0u : 8u);
    if (bad != 0u) {  // reported, not written
      if (lane == 0 && P.status != nullptr) atomicOr(P.status, bad);
      return;
    }
    norm_rope_row_by(P.kv_raw + (int64_t)t * P.kv_row_stride, P.kv_weight, P.kv_eps, angle, row_width(P.layout), lane,
                     srow[wi]);
    write_any_row(srow[wi], lane, P.kv, P.layout, page, slot & (P.page_size - 1), P.page_size, P.page_bytes);
    return;
  }
  const int groups = (P.heads + per - 1) / per;  // of heads
  const int64_t w = static_cast<int64_t>(blockIdx.x - P.kv_blocks) * kAxesWarps + wi;
  if (w >= static_cast<int64_t>(P.tokens) * groups) return;
  const int t = static_cast<int>(w / groups);
  const int n0 = static_cast<int>(w - static_cast<int64_t>(t) * groups) * per, n1 = min(n0 + per, P.heads);
  const Angles angle(A, t);
  if (!angle.ok) {  // left as it was; reported unless it is padding
    if (lane == 0 && P.status != nullptr && !(angle.below && P.slots[t] < 0)) atomicOr(P.status, 8u);
    return;
  }
  const uint16_t* qn = P.q_nope + t * P.nope_token_stride;
  const uint16_t* qp = P.q_pe + t * P.pe_token_stride;
  uint16_t* q = P.q_out + static_cast<int64_t>(t) * P.heads * WIDTH;

  if (WIDTH == 192) {
    // four heads a step: 4 x 16 chunks of 16 bytes of the NoPE parts, two a lane, and 4 x 8 of the RoPE parts
    const int c = lane & 7;
    float2 cs[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) cs[k] = angle(4 * c + k);
#pragma unroll 2
    for (int n = n0; n < n1; n += 4) {
      const int h0 = n + (lane >> 4), h1 = h0 + 2, hp = n + (lane >> 3);
      uint4 u0, u1, up;
      if (A.copy_nope) {
        if (h0 < n1) u0 = reinterpret_cast<const uint4*>(qn + h0 * P.nope_head_stride)[lane & 15];
        if (h1 < n1) u1 = reinterpret_cast<const uint4*>(qn + h1 * P.nope_head_stride)[lane & 15];
      }
      if (hp < n1) up = reinterpret_cast<const uint4*>(qp + hp * P.pe_head_stride)[c];
      if (A.copy_nope) {
        if (h0 < n1) reinterpret_cast<uint4*>(q + h0 * WIDTH)[lane & 15] = u0;
        if (h1 < n1) reinterpret_cast<uint4*>(q + h1 * WIDTH)[lane & 15] = u1;
      }
      if (hp < n1)
        reinterpret_cast<uint4*>(q + hp * WIDTH + 128)[c] =
            make_uint4(rotate2(up.x, cs[0]), rotate2(up.y, cs[1]), rotate2(up.z, cs[2]), rotate2(up.w, cs[3]));
    }
    return;
  }

  // 64 chunks of 16 bytes, two a lane, normalised over their 512 elements where asked; the 576-wide rows' RoPE part is
  // a pair a lane, that of the 512-wide rows the last eight chunks
  const bool pe_lane = WIDTH == 512 && lane >= 24;
  float2 cs[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    cs[k] = WIDTH == 576 ? (k == 0 ? angle(lane) : make_float2(1.f, 0.f)) : angle(4 * (lane & 7) + k);
  for (int n = n0; n < n1; ++n) {
    const uint16_t* an = qn + n * P.nope_head_stride;
    const uint16_t* ap = qp + n * P.pe_head_stride;
    const uint4 u0 = *reinterpret_cast<const uint4*>(an + 8 * lane);
    const uint4 u1 = *reinterpret_cast<const uint4*>(pe_lane ? ap + 8 * (lane - 24) : an + 256 + 8 * lane);
    uint32_t two = 0;
    if (WIDTH == 576) two = reinterpret_cast<const uint32_t*>(ap)[lane];
    uint4 o0 = u0, o1 = u1;
    if (WIDTH == 512 || P.q_norm) {  // (a bf16 value goes through fp32 unchanged)
      float a[8], b[8];
      unpack8(u0, a);
      unpack8(u1, b);
      if (P.q_norm) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(a[k], a[k], fmaf(b[k], b[k], ss));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rinv = 1.0f / sqrtf(ss * (1.0f / 512.0f) + P.q_eps);
        float wa[8], wb[8];
        if (P.q_weight != nullptr) {
          unpack8(reinterpret_cast<const uint4*>(P.q_weight)[lane], wa);
          unpack8(reinterpret_cast<const uint4*>(P.q_weight)[32 + lane], wb);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          a[k] *= rinv;
          b[k] *= rinv;
          if (P.q_weight != nullptr) {
            a[k] *= wa[k];
            b[k] *= wb[k];
          }
        }
      }
      if (pe_lane) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x0 = b[2 * k], x1 = b[2 * k + 1];
          b[2 * k] = x0 * cs[k].x - x1 * cs[k].y;
          b[2 * k + 1] = x0 * cs[k].y + x1 * cs[k].x;
        }
      }
      o0 = pack8(a);
      o1 = pack8(b);
    }
    uint16_t* o = q + n * WIDTH;
    if (A.copy_nope || WIDTH == 512) {
      reinterpret_cast<uint4*>(o)[lane] = o0;
      reinterpret_cast<uint4*>(o)[32 + lane] = o1;
    }
    if (WIDTH == 576) reinterpret_cast<uint32_t*>(o + 512)[lane] = rotate2(two, cs[0]);
  }
}

}  // namespace

cudaError_t launch_qkv_norm_rope_axes(const AxesParams& p, cudaStream_t stream) {
  AxesParams a = p;
  a.qkv.kv_blocks = (p.qkv.tokens + kAxesWarps - 1) / kAxesWarps;
  const int per = p.q_width == 192 ? 8 : 1;
  const int64_t warps = static_cast<int64_t>(p.qkv.tokens) * ((p.qkv.heads + per - 1) / per);
  const dim3 grid(static_cast<unsigned>(a.qkv.kv_blocks + (warps + kAxesWarps - 1) / kAxesWarps)), block(kAxesWarps * 32);
  if (p.q_width == 192) return launch_pdl(axes_kernel<192>, grid, block, 0, stream, a, per);
  if (p.q_width == 576) return launch_pdl(axes_kernel<576>, grid, block, 0, stream, a, per);
  return launch_pdl(axes_kernel<512>, grid, block, 0, stream, a, per);
}

}  // namespace mla
