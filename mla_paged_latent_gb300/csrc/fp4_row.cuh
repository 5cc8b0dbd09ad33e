// The 4-bit row: e2m1 codes with one ue8m0 scale per 32 elements, decoded to bf16 and encoded
// from fp32. Shared by the decode kernel, the KV writes and the reads back.
//
// e2m1 (OCP MX): sign, two exponent bits (bias 1), one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6.
// A value is e2m1(code) * 2^(scale - 127); a code has two significant bits, so the product is
// exact in bf16 (subnormals included) unless it overflows. Element 2i of a row is the low
// nibble of byte i, element 2i + 1 the high one.
#pragma once
#include <cstdint>

#include "ptx_sm103.cuh"

namespace mla {

constexpr int kFp4Group = 32;         // elements that share a scale
constexpr int kFp4ScaleSlot = 16;     // bytes of a row's scale slot

// ue8m0 byte -> the bf16 pair (2^(b - 127), 2^(b - 127)); 0 is the subnormal 2^-127, 255 NaN.
__device__ __forceinline__ uint32_t ue8m0_to_bf16x2(uint32_t b) {
  const uint32_t h = b == 0u ? 0x0040u : (b == 255u ? 0x7FC0u : b << 7);
  return h * 0x00010001u;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight codes (element 0 in bits 0-3) times the scale pair -> four bf16 pairs in element order.
// The magnitudes' high and low bytes come from two 8-entry tables, four codes a byte permute (the
// codes' own nibbles are the selectors), the sign bits are spread into the high bytes, and two more
// permutes interleave them: 2.6 instructions an element pair with the exact product, against 4 for
// a conversion through f16 and fp32.
__device__ __forceinline__ void fp4x8_to_bf16(uint32_t w, uint32_t scale2, uint32_t (&o)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t v = h ? w >> 16 : w;
    const uint32_t sel = v & 0x7777u;
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
    uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel);
    const uint32_t s = __byte_perm(v, 0u, 0x1100);  // bytes 0, 0, 1, 1: two codes in each
    hi |= s & 0x80008000u;
    hi |= (s << 4) & 0x00800080u;
    o[2 * h] = mul_bf16x2(__byte_perm(lo, hi, 0x5140), scale2);
    o[2 * h + 1] = mul_bf16x2(__byte_perm(lo, hi, 0x7362), scale2);
  }
}

// 6 * 2^e as fp32 (exact; +inf once it exceeds the fp32 range).
__device__ __forceinline__ float pow2x6(int e) {
  const int E = e + 2 + 127;  // 6 = 1.5 * 2^2
  if (E >= 255) return __uint_as_float(0x7F800000u);
  if (E <= 0) return 0.f;
  return __uint_as_float((static_cast<uint32_t>(E) << 23) | 0x400000u);
}
// Smallest e with 6 * 2^e >= a (a >= 1e-10), clamped to [-127, 127].
__device__ __forceinline__ int fp4_group_exponent(float a) {
  if (!(a <= 3.4028235e38f)) return 127;
  int e = static_cast<int>((__float_as_uint(a) >> 23) & 0xFFu) - 127 - 2;
  if (!(pow2x6(e) >= a)) ++e;  // a's mantissa is above 1.5
  return e > 127 ? 127 : e;
}
// Two fp32 -> two e2m1 codes, to nearest even, saturating; `lo` in bits 0-3, `hi` in bits 4-7.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace mla
