// KV rows, one warp each: the layouts' geometry, the quantising write of a bf16 row into its
// page slot, and the RMSNorm + RoPE that precede it. Shared by the plain write, the fused write
// and the step that prepares queries and KV rows together, so that all three write the same bytes.
#pragma once
#include <cstdint>

#include "fp4_row.cuh"
#include "mla_kernels.h"
#include "ptx_sm103.cuh"

namespace mla {

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

// Geometry of a stored row: NoPE elements, bytes of the row, bytes of its scale slot, and
// elements of the bf16 row that a write takes (K's width).
__host__ __device__ constexpr int row_nope(int layout) { return layout == 1 || layout == 3 ? 448 : 512; }
__host__ __device__ constexpr int row_stored_bytes(int layout) {
  return layout == 0 ? 1152 : layout == 1 ? 576 : layout == 2 ? 640 : layout == 3 ? 352 : 384;
}
__host__ __device__ constexpr int row_scale_slot(int layout) { return layout == 0 ? 0 : layout <= 2 ? 8 : kFp4ScaleSlot; }
__host__ __device__ constexpr int row_width(int layout) { return layout == 1 || layout == 3 ? 512 : 576; }

// 448 * 2^e as fp32 (exact; +inf once it exceeds the fp32 range).
__device__ __forceinline__ float pow2x448(int e) {
  const int E = e + 8 + 127;  // 448 = 1.75 * 2^8
  if (E >= 255) return __uint_as_float(0x7F800000u);
  if (E <= 0) return 0.f;
  return __uint_as_float((static_cast<uint32_t>(E) << 23) | 0x600000u);
}
// Smallest e with 448 * 2^e >= a (a >= 1e-10), clamped to [-127, 127]; decided by
// exact comparisons of powers of two.
__device__ __forceinline__ int group_exponent(float a) {
  if (!(a <= 3.4028235e38f)) return 127;
  int e = static_cast<int>((__float_as_uint(a) >> 23) & 0xFFu) - 127 - 8;
  while (e < 127 && !(pow2x448(e) >= a)) ++e;
  while (e > -127 && pow2x448(e - 1) >= a) --e;
  return e;
}
// 2^-e as fp32 (exact for e in [-127, 126]).
__device__ __forceinline__ float pow2neg(int e) {
  const int E = 127 - e;
  if (E >= 255) return __uint_as_float(0x7F800000u);
  if (E <= 0) return __uint_as_float(0x00400000u >> (-E));
  return __uint_as_float(static_cast<uint32_t>(E) << 23);
}

// The 4-bit form of write_row: lane l holds elements [16 l, 16 l + 16) of the bf16 row in x0 and x1, and lanes 0-7 the
// RoPE part's elements [8 l, 8 l + 8) in pe. A group is lanes 2g and 2g + 1. Codes are rounded to nearest even after an
// exact product with a power of two (what that takes below bf16's range is far below half a code). e2m1 has no
// NaN: a group that holds one gets the scale byte 255 (NaN) and zero codes, so that it reads back as NaN.
__device__ __forceinline__ void write_row_fp4(uint4 x0, uint4 x1, uint4 pe, int lane, int nope, uint8_t* dst,
                                              uint8_t* slot) {
  const uint32_t h[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  uint32_t m = 0;  // magnitudes compare as integers, NaN above infinity
#pragma unroll
  for (int k = 0; k < 8; ++k) m = __vmaxu2(m, h[k] & 0x7FFF7FFFu);
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t sbyte = fp4_scale_byte(m >> 16 > (m & 0xFFFFu) ? m >> 16 : m & 0xFFFFu);
  if (lane * 16 < nope) {
    // 2^-e as a bf16 pair: exponent field 254 - (e + 127); 2^-127, an infinity's, is subnormal
    const uint32_t sc = (sbyte < 254u ? (254u - sbyte) << 7 : 0x40u) * 0x00010001u;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t p = mul_bf16x2(h[4 * i + k], sc);
        v[2 * k] = __uint_as_float(p << 16);
        v[2 * k + 1] = __uint_as_float(p & 0xFFFF0000u);
      }
      w[i] = sbyte == 255u ? 0u : f32x8_to_e2m1x8(v);
    }
    reinterpret_cast<uint2*>(dst)[lane] = make_uint2(w[0], w[1]);
  }
  // the 64 RoPE elements stay bf16, after the codes
  if (lane < 8) reinterpret_cast<uint4*>(dst + nope / 2)[lane] = pe;
  // scale bytes: group g's sits in lanes 2g and 2g + 1; zeros behind the last
  if ((lane & 1) == 0) slot[lane >> 1] = lane * 16 < nope ? static_cast<uint8_t>(sbyte) : 0;
}

// Write one bf16 row (generic pointer x, 16-byte aligned, row_elems values) into its
// page slot (layouts of 8 and 16 bits); all 32 lanes of the warp take part ("MLA" API page of HALOps,
// mla_attention: KV cache write of the RMSNorm'd row; kv_cache parameter for the layout).
__device__ __forceinline__ void write_row(const uint16_t* x, int lane, uint8_t* kv, int layout,
                                          int64_t page, int off, int page_size, int64_t page_bytes) {
  if (layout == 0) {
    const uint4* src = reinterpret_cast<const uint4*>(x);
    uint4* dst = reinterpret_cast<uint4*>(kv + page * page_bytes + (int64_t)off * 1152);
    const uint4 c0 = src[lane], c1 = src[32 + lane], c2 = src[64 + (lane & 7)];
    dst[lane] = c0;
    dst[32 + lane] = c1;
    if (lane < 8) dst[64 + lane] = c2;
    return;
  }
  const int nope = row_nope(layout);
  const int row_bytes = row_stored_bytes(layout);
  uint8_t* dst = kv + page * page_bytes + (int64_t)off * row_bytes;
  // lane l holds elements [16 l, 16 l + 16), loaded at once; NoPE group g is lanes 4g .. 4g+3
  // (in the 512-wide DSV4 rows, lanes 28-31 hold the RoPE part)
  const uint4 x0 = reinterpret_cast<const uint4*>(x)[2 * lane];
  const uint4 x1 = reinterpret_cast<const uint4*>(x)[2 * lane + 1];
  uint4 pe = make_uint4(0, 0, 0, 0);  // the 576-wide row's RoPE part
  if (layout != 1 && lane < 8) pe = reinterpret_cast<const uint4*>(x + nope)[lane];
  float v[16];
  {
    const uint32_t h[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[2 * k] = bf16_to_f32(h[k] & 0xFFFFu);
      v[2 * k + 1] = bf16_to_f32(h[k] >> 16);
    }
  }
  const bool in_nope = lane * 16 < nope;
  float a = 0.f;  // fmaxf returns the number when one operand is NaN: NaN elements do not count
#pragma unroll
  for (int k = 0; k < 16; ++k) a = fmaxf(a, fabsf(v[k]));
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
  a = fmaxf(a, 1e-10f);
  const int e = group_exponent(a);
  if (in_nope) {
    const float sc = pow2neg(e);
    uint32_t w4[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint16_t c0, c1;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c0) : "f"(v[4 * k + 1] * sc), "f"(v[4 * k] * sc));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c1) : "f"(v[4 * k + 3] * sc), "f"(v[4 * k + 2] * sc));
      w4[k] = static_cast<uint32_t>(c0) | (static_cast<uint32_t>(c1) << 16);
      // a NaN element (left out of the amax above) is stored as the NaN code 0x7F, whatever its sign
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (v[4 * k + b] != v[4 * k + b]) w4[k] = (w4[k] & ~(0xFFu << (8 * b))) | (0x7Fu << (8 * b));
    }
    reinterpret_cast<uint4*>(dst)[lane] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
  } else {
    // DSV4 row: its 64 RoPE elements stay bf16, after the 448 code bytes
    uint4* d2 = reinterpret_cast<uint4*>(dst + nope + (lane * 16 - nope) * 2);
    d2[0] = x0;
    d2[1] = x1;
  }
  // scale bytes: group g's exponent sits in lane 4g; lane 0 assembles the 8-byte slot
  uint32_t sbytes[2] = {0u, 0u};
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const int eg = __shfl_sync(0xffffffffu, e, 4 * g);
    if (g < nope / 64) sbytes[g >> 2] |= static_cast<uint32_t>(eg + 127) << (8 * (g & 3));
  }
  if (layout != 1 && lane < 8) reinterpret_cast<uint4*>(dst + nope)[lane] = pe;
  if (lane == 0) {
    uint2* sp = reinterpret_cast<uint2*>(kv + page * page_bytes + (int64_t)page_size * row_bytes + off * 8);
    *sp = make_uint2(sbytes[0], sbytes[1]);
  }
}

// write_row for every layout.
__device__ __forceinline__ void write_any_row(const uint16_t* x, int lane, uint8_t* kv, int layout,
                                              int64_t page, int off, int page_size, int64_t page_bytes) {
  if (layout < 3) {
    write_row(x, lane, kv, layout, page, off, page_size, page_bytes);
    return;
  }
  const int nope = row_nope(layout), row_bytes = row_stored_bytes(layout);
  const uint4* src = reinterpret_cast<const uint4*>(x);
  uint8_t* const pg = kv + page * page_bytes;
  write_row_fp4(src[2 * lane], src[2 * lane + 1], src[nope / 8 + (lane & 7)], lane, nope, pg + (int64_t)off * row_bytes,
                pg + (int64_t)page_size * row_bytes + (int64_t)off * kFp4ScaleSlot);
}

// RMSNorm of the 512 latent elements and RoPE of the 64 RoPE elements of one raw row x
// (16-byte aligned), in fp32, rounded once to bf16 into srow (shared memory; all lanes of the warp
// take part, and it ends with a __syncwarp). Lane l holds latent elements [16 l, 16 l + 16) and
// RoPE pair l of the 576-wide layouts; f is the position's row of the (cos, sin) table.
__device__ __forceinline__ void norm_rope_row(const uint16_t* x, const uint16_t* w, float eps,
                                              const float* f, int width, int lane, uint16_t* srow) {
  float v[16];
  {
    const uint4 a = reinterpret_cast<const uint4*>(x)[2 * lane];
    const uint4 b = reinterpret_cast<const uint4*>(x)[2 * lane + 1];
    const uint32_t h[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[2 * k] = bf16_to_f32(h[k] & 0xFFFFu);
      v[2 * k + 1] = bf16_to_f32(h[k] >> 16);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) ss = fmaf(v[k], v[k], ss);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float rinv = 1.0f / sqrtf(ss * (1.0f / 512.0f) + eps);
  {
    const uint4 a = reinterpret_cast<const uint4*>(w)[2 * lane];
    const uint4 b = reinterpret_cast<const uint4*>(w)[2 * lane + 1];
    const uint32_t h[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[2 * k] = v[2 * k] * rinv * bf16_to_f32(h[k] & 0xFFFFu);
      v[2 * k + 1] = v[2 * k + 1] * rinv * bf16_to_f32(h[k] >> 16);
    }
  }
  if (width == 512 && lane >= 28) {
    // 512-wide row: elements 448..511 (lanes 28-31) are the RoPE part, rotated after the norm
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = 8 * (lane - 28) + k;
      const float c = f[2 * i], s = f[2 * i + 1];
      const float x0 = v[2 * k], x1 = v[2 * k + 1];
      v[2 * k] = x0 * c - x1 * s;
      v[2 * k + 1] = x0 * s + x1 * c;
    }
  }
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = f32x2_to_bf16x2(v[2 * k], v[2 * k + 1]);
  reinterpret_cast<uint4*>(srow)[2 * lane] = make_uint4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<uint4*>(srow)[2 * lane + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  if (width != 512) {
    // k_pe (elements 512..575) is rotated as it comes, without the norm
    const uint32_t two = reinterpret_cast<const uint32_t*>(x + 512)[lane];
    const float x0 = bf16_to_f32(two & 0xFFFFu), x1 = bf16_to_f32(two >> 16);
    const float c = f[2 * lane], s = f[2 * lane + 1];
    reinterpret_cast<uint32_t*>(srow + 512)[lane] = f32x2_to_bf16x2(x0 * c - x1 * s, x0 * s + x1 * c);
  }
  __syncwarp();
}

}  // namespace mla
