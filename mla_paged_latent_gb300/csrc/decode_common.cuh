// Device helpers shared by the decode kernels: the unit schedule of a
// split-KV partition and the base-2 exponential.
#pragma once
#include <cstdint>

#include "mla_kernels.h"
#include "ptx_sm103.cuh"

namespace mla {

__device__ __forceinline__ int num_blocks(const DecodeParams& P, int r) {
  const int K = P.topk > 0 ? P.topk : P.seqlens[r];
  const int nb = (K + kBlockRows - 1) / kBlockRows;
  return nb < 1 ? 1 : nb;
}

// Segments (request, block range, split index) of one partition, in order.
template <typename F>
__device__ __forceinline__ void for_each_unit(const DecodeParams& P, int part, F&& f) {
  const int* s = P.sched + 8 * part;
  const int b0 = s[0], k0 = s[1], b1 = s[2], k1 = s[3], fs = s[4];
  for (int r = b0; r < P.batch && (r < b1 || (r == b1 && k1 > 0)); ++r) {
    const int nb = num_blocks(P, r);
    const int lo = (r == b0) ? k0 : 0;
    const int hi = (r == b1) ? (k1 < nb ? k1 : nb) : nb;
    if (hi <= lo) continue;
    f(r, lo, hi, (r == b0) ? fs : 0);
  }
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// the largest of three; a NaN gives way to a number
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
__device__ __forceinline__ float2 fma2v(float2 a, float2 b, float2 c) {  // a b + c, lane by lane
  float2 r;
  asm("{\n .reg .b64 p, q, s, d;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n mov.b64 s, {%6, %7};\n"
      " fma.rn.f32x2 d, p, q, s;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
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

// mbar_wait (and mbar_wait_cluster) in few instructions, bounded the same way. The roles of a CTA run at once from
// one instruction cache, and those functions inlined at each wait were a third of the 4-bit pair kernel's code
// (instruction fetches were a sixth of all stalls; a call instead costs the registers that live across it: 132 us
// against 140). No timer is read before the first test has failed, and the tests carry no suspend hint (each 1%).
__device__ __forceinline__ bool wait_bar(uint32_t b, uint32_t parity, volatile int* abort, unsigned int* status) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u64 t0, t;\n .reg .u32 a;\n"
      " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n @p bra DONE_%=;\n"
      " mov.u64 t0, %%globaltimer;\n"
      "POLL_%=:\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n @p bra DONE_%=;\n"
      " ld.volatile.shared.u32 a, [%3];\n mov.u64 t, %%globaltimer;\n sub.u64 t, t, t0;\n"
      " setp.lt.u64 q, t, 2000000000;\n setp.eq.and.u32 q, a, 0, q;\n @q bra POLL_%=;\n"
      "DONE_%=:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(b), "r"(parity), "r"(smem_addr(const_cast<int*>(abort)))
      : "memory");
  if (ok != 0) return true;
  if (*abort == 0) {
    atomicOr(status, 1u);
    *abort = 1;
  }
  return false;
}

}  // namespace mla
