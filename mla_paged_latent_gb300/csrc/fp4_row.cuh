// The 4-bit row: e2m1 codes with one ue8m0 scale per 32 elements, decoded to bf16 and encoded
// from it. Shared by the decode kernels, the KV writes and the reads back.
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

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A group's scale 2^(b - 127) in two factors: f16 bits, which hold 2^-14 .. 2^15, and a bf16 pair with the
// rest (one for the scales of ordinary rows; NaN for b = 255).
struct Fp4Scale {
  uint16_t h;
  uint32_t rest;
};
__device__ __forceinline__ bool fp4_scale_plain(uint32_t b) { return b - 113u <= 29u; }  // rest is one
__device__ __forceinline__ Fp4Scale fp4_scale(uint32_t b) {
  const uint32_t c = b < 113u ? 113u : (b > 142u ? 142u : b);
  Fp4Scale s;
  s.h = static_cast<uint16_t>((c - 112u) << 10);
  s.rest = b == 255u ? 0x7FC07FC0u : ((b + 127u - c) << 7) * 0x00010001u;
  return s;
}
// Eight codes (element 0 in bits 0-3) times the scale -> four bf16 pairs in element order, exactly: e2m1 to f16,
// an fp32 product with the f16 factor, two of them rounded (that is, cut) to a bf16 pair. Measured for a group
// of 32 a lane, on all four sub-partitions, with the 64 bytes stored: 93 cycles; with the magnitudes taken from
// byte-permute tables and the signs joined on, which all runs in one pipe, 130; a plain f16 product, which loses
// scales, 74, where the stores are the bound. (The -0.0 addend keeps the sign of a zero.) PLAIN: the caller has seen
// that the rest is one.
template <bool PLAIN = false>
__device__ __forceinline__ void fp4x8_to_bf16(uint32_t w, const Fp4Scale& s, uint32_t (&o)[4]) {
  uint32_t h[4];
  asm("{\n .reg .b8 t0, t1, t2, t3;\n mov.b32 {t0, t1, t2, t3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, t0;\n cvt.rn.f16x2.e2m1x2 %1, t1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, t2;\n cvt.rn.f16x2.e2m1x2 %3, t3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n fma.rn.f32.f16 %0, l, %3, %4;\n fma.rn.f32.f16 %1, u, %3, %4;\n}\n"
        : "=f"(a), "=f"(b)
        : "r"(h[i]), "h"(s.h), "f"(-0.0f));
    o[i] = f32x2_to_bf16x2(a, b);
  }
  if (!PLAIN) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mul_bf16x2(o[i], s.rest);
  }
}

// The scale byte e + 127 of a group whose largest magnitude has the bf16 bits m (taken as integers, so that a NaN
// counts as the largest): the smallest e with 6 * 2^e >= max(m, 1e-10), where 6 = 1.5 * 2^2; 254 for an infinity, 255
// for a NaN.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t m) {
  const uint32_t e = (m >> 7) - ((m & 0x7Fu) > 0x40u ? 1u : 2u);  // negative below 2^-125: the lower bound takes it
  const uint32_t f = static_cast<int>(e) < 92 ? 92u : e;          // 1e-10 = 1.718 * 2^-34: e = -35
  return m < 0x7F80u ? f : (m == 0x7F80u ? 254u : 255u);
}
// Eight fp32 -> eight e2m1 codes, to nearest even, saturating; element 0 in bits 0-3.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

}  // namespace mla
