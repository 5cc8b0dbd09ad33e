// The steps around a cache that the decode reads: queries and new KV rows normalised, rotated and
// put in place in one launch, and cached rows read back as bf16.
#include <cstdint>
#include <cuda_runtime.h>

#include "kv_row.cuh"
#include "mla_kernels.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

constexpr int kRowWarps = 8;  // rows per block, one warp each

// ----------------------------------------------------------------------------- queries and KV rows
// 16 bytes (8 elements) of a query row held by a lane, times their norm factor and gain.
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

// One warp per row. The first blocks take the KV rows (norm_rope_row + write_any_row, as the
// fused write), the others the (token, head) query rows: 64 sixteen-byte chunks, two a lane, NoPE from
// q_nope and (512-wide rows) RoPE from q_pe, normalised over all 512 elements when asked; the
// 576-wide rows' RoPE part is one pair a lane, rotated as it comes. A row is read whole into
// registers before any of it is written, so q may be prepared in place. Bound by the bytes (2.3 KB a query row), and
// for those by the loads in flight: 8192 x 128 rows of 576 take 366 us at eight blocks an SM (32 registers a thread,
// some of the KV rows' spilled; 6.7 TB/s, as fast as a copy), 401 at six, 426 at five (48 registers).
template <int WIDTH>
__global__ void __launch_bounds__(kRowWarps * 32, 8) qkv_norm_rope_kernel(const __grid_constant__ QkvParams P) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) uint16_t srow[kRowWarps][576];
  const int wi = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) < P.kv_blocks) {
    const int r = blockIdx.x * kRowWarps + wi;
    if (r >= P.tokens) return;
    const int slot = P.slots[r];
    if (slot < 0) return;
    const int page = slot >> (31 - __clz(P.page_size));  // (a power of two)
    const int pos = P.positions[r];
    const uint32_t bad = (page >= P.num_pages ? 4u : 0u) | (pos < 0 || pos >= P.max_pos ? 8u : 0u);
    if (bad != 0u) {  // reported, not written
      if (lane == 0 && P.status != nullptr) atomicOr(P.status, bad);
      return;
    }
    norm_rope_row(P.kv_raw + (int64_t)r * P.kv_row_stride, P.kv_weight, P.kv_eps, P.freqs + (int64_t)pos * 64, WIDTH,
                  lane, srow[wi]);
    write_any_row(srow[wi], lane, P.kv, P.layout, page, slot & (P.page_size - 1), P.page_size, P.page_bytes);
    return;
  }
  // (the entry point keeps tokens * heads below 2^31, and a block's rows end at most 7 past it)
  const uint32_t row = (blockIdx.x - P.kv_blocks) * kRowWarps + wi;
  if (row >= static_cast<uint32_t>(P.tokens) * P.heads) return;
  const int t = static_cast<int>(row / static_cast<uint32_t>(P.heads));
  const int n = static_cast<int>(row) - t * P.heads;
  const int pos = P.positions[t];
  if (pos < 0 || pos >= P.max_pos) {  // left as it was; reported unless it is padding
    if (lane == 0 && P.status != nullptr && (pos >= 0 || P.slots[t] >= 0)) atomicOr(P.status, 8u);
    return;
  }
  const uint16_t* qn = P.q_nope + t * P.nope_token_stride + n * P.nope_head_stride;
  const uint16_t* qp = P.q_pe + t * P.pe_token_stride + n * P.pe_head_stride;
  const float* f = P.freqs + (int64_t)pos * 64;
  const bool pe_lane = WIDTH == 512 && lane >= 24;  // its second chunk is RoPE pairs 4 (lane - 24) ..
  const uint4 u0 = *reinterpret_cast<const uint4*>(qn + 8 * lane);
  const uint4 u1 = *reinterpret_cast<const uint4*>(pe_lane ? qp + 8 * (lane - 24) : qn + 256 + 8 * lane);
  uint32_t two = 0;
  float2 cs = make_float2(0.f, 0.f);
  if (WIDTH == 576) {
    two = reinterpret_cast<const uint32_t*>(qp)[lane];
    cs = reinterpret_cast<const float2*>(f)[lane];
  }
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
      if (P.q_weight != nullptr) {
        float wa[8], wb[8];
        unpack8(reinterpret_cast<const uint4*>(P.q_weight)[lane], wa);
        unpack8(reinterpret_cast<const uint4*>(P.q_weight)[32 + lane], wb);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          a[k] = a[k] * rinv * wa[k];
          b[k] = b[k] * rinv * wb[k];
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          a[k] *= rinv;
          b[k] *= rinv;
        }
      }
    }
    if (pe_lane) {
      const float4* f4 = reinterpret_cast<const float4*>(f) + 2 * (lane - 24);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 c = f4[k];
        const float x0 = b[4 * k], x1 = b[4 * k + 1], x2 = b[4 * k + 2], x3 = b[4 * k + 3];
        b[4 * k] = x0 * c.x - x1 * c.y;
        b[4 * k + 1] = x0 * c.y + x1 * c.x;
        b[4 * k + 2] = x2 * c.z - x3 * c.w;
        b[4 * k + 3] = x2 * c.w + x3 * c.z;
      }
    }
    o0 = pack8(a);
    o1 = pack8(b);
  }
  uint16_t* q = P.q_out + (int64_t)row * WIDTH;
  reinterpret_cast<uint4*>(q)[lane] = o0;
  reinterpret_cast<uint4*>(q)[32 + lane] = o1;
  if (WIDTH == 576) {
    const float x0 = bf16_to_f32(two & 0xFFFFu), x1 = bf16_to_f32(two >> 16);
    reinterpret_cast<uint32_t*>(q + 512)[lane] = f32x2_to_bf16x2(x0 * cs.x - x1 * cs.y, x0 * cs.y + x1 * cs.x);
  }
}

// ----------------------------------------------------------------------------- read back
// One warp per row: the cached row at slots[r], decoded to bf16. A lane takes eight elements a
// step, so loads and stores of a warp are contiguous.
template <int LAYOUT>
__global__ void __launch_bounds__(kRowWarps * 32) kv_read_kernel(const uint8_t* kv, int64_t num_pages,
                                                                 int page_size, int64_t page_bytes,
                                                                 const int32_t* slots, int n,
                                                                 uint16_t* out, uint32_t* status) {
  pdl_trigger();
  pdl_wait();
  constexpr int kNope = row_nope(LAYOUT), kRowBytes = row_stored_bytes(LAYOUT), kWidth = row_width(LAYOUT);
  constexpr int kCodeBytes = LAYOUT == 0 ? 1024 : LAYOUT <= 2 ? kNope : kNope / 2;
  const int r = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= n) return;
  const int slot = slots[r];
  if (slot < 0) return;
  const int page = slot >> (31 - __clz(page_size));  // (a power of two)
  const int off = slot & (page_size - 1);
  if (page >= num_pages) {  // reported, not read
    if (lane == 0 && status != nullptr) atomicOr(status, 4u);
    return;
  }
  const uint8_t* src = kv + page * page_bytes + (int64_t)off * kRowBytes;
  const uint8_t* sc = kv + page * page_bytes + (int64_t)page_size * kRowBytes + (int64_t)off * row_scale_slot(LAYOUT);
  uint4* dst = reinterpret_cast<uint4*>(out + (int64_t)r * kWidth);
  // every load before the first store, which may alias them for all that the compiler knows
  uint4 pe = make_uint4(0, 0, 0, 0);
  if (lane < 8) pe = reinterpret_cast<const uint4*>(src + kCodeBytes)[lane];
  uint4 raw[2];      // elements 8c .. 8c + 7, c = lane + 32 h: 16, 8 or 4 bytes
  uint32_t sb[2];    // and their scale byte
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = lane + 32 * h;
    if (8 * c >= kNope) break;
    if (LAYOUT == 0) {
      raw[h] = reinterpret_cast<const uint4*>(src)[c];
    } else if (LAYOUT <= 2) {
      const uint2 w = reinterpret_cast<const uint2*>(src)[c];
      raw[h] = make_uint4(w.x, w.y, 0, 0);
      sb[h] = sc[c >> 3];
    } else {
      raw[h] = make_uint4(reinterpret_cast<const uint32_t*>(src)[c], 0, 0, 0);
      sb[h] = sc[c >> 2];
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = lane + 32 * h;
    if (8 * c >= kNope) break;
    if (LAYOUT == 0) {
      dst[c] = raw[h];
    } else if (LAYOUT <= 2) {
      const float s = ue8m0_to_f32(sb[h]);
      const float2 a = e4m3x2_to_f32x2(raw[h].x & 0xFFFFu), b = e4m3x2_to_f32x2(raw[h].x >> 16);
      const float2 d = e4m3x2_to_f32x2(raw[h].y & 0xFFFFu), e = e4m3x2_to_f32x2(raw[h].y >> 16);
      dst[c] = make_uint4(f32x2_to_bf16x2(a.x * s, a.y * s), f32x2_to_bf16x2(b.x * s, b.y * s),
                          f32x2_to_bf16x2(d.x * s, d.y * s), f32x2_to_bf16x2(e.x * s, e.y * s));
    } else {
      uint32_t o[4];
      fp4x8_to_bf16(raw[h].x, fp4_scale(sb[h]), o);
      dst[c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (lane < 8) dst[kNope / 8 + lane] = pe;
}

}  // namespace

cudaError_t launch_qkv_norm_rope(const QkvParams& p, cudaStream_t stream) {
  QkvParams q = p;
  q.kv_blocks = (p.tokens + kRowWarps - 1) / kRowWarps;
  const int64_t rows = static_cast<int64_t>(p.tokens) * p.heads;
  const dim3 grid(static_cast<unsigned>(q.kv_blocks + (rows + kRowWarps - 1) / kRowWarps));
  return row_width(p.layout) == 512 ? launch_pdl(qkv_norm_rope_kernel<512>, grid, dim3(kRowWarps * 32), 0, stream, q)
                                    : launch_pdl(qkv_norm_rope_kernel<576>, grid, dim3(kRowWarps * 32), 0, stream, q);
}

cudaError_t launch_kv_read(const uint8_t* kv, int layout, int64_t num_pages, int page_size, int64_t page_bytes,
                           const int32_t* slots, int n, uint16_t* out, uint32_t* status, cudaStream_t stream) {
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3((n + kRowWarps - 1) / kRowWarps), dim3(kRowWarps * 32), 0, stream, kv, num_pages,
                      page_size, page_bytes, slots, n, out, status);
  };
  switch (layout) {
    case 0: return go(kv_read_kernel<0>);
    case 1: return go(kv_read_kernel<1>);
    case 2: return go(kv_read_kernel<2>);
    case 3: return go(kv_read_kernel<3>);
    default: return go(kv_read_kernel<4>);
  }
}

}  // namespace mla
