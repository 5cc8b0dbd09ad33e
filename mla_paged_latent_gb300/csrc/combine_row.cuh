// The merge of one query row's split-KV partials, shared by the combine kernel and the
// fused combine + value up-projection so that both write the same merged rows.
#pragma once
#include <cstdint>

#include "ptx_sm103.cuh"

namespace mla {

// Warp-wide, one query row `row` of a request with ns >= 2 partials starting at split s0:
// lse = ln sum_s e^(lse_s); out = sum_s e^(lse_s - lse) o_s ("mla_attention.py ·
// tduncan/Nvidia-Optimization-Stack-VLLM", Chunked Prefill: merge_attn_states; an empty
// partial has lse = -inf and weight 0), then the sink factor 1 / (1 + e^(sink - lse))
// ("MLA" API page of HALOps, mla_output_proj: the split-KV LSE combine receives attn_sink).
// acc[4 k + i] receives element 4 (32 (k0 + k) + lane) + i: the whole row (N = 16), or a quarter
// of it (N = 4, k0 = 0 .. 3); the return value is lse (-inf, with acc = 0, when every partial is
// empty). A partial whose lse is NaN is not empty and makes NaN of lse and acc; the maximum passes
// over it, so what is empty is asked of the partials themselves.
// U partials of more than four are loaded at once (the fused up-projection takes U = 1: 121 registers instead of 128 and
// spills, 24.0 us against 25.6 on 128 requests of two partials, 63.6 against 68.7 on 512 of one).
template <int N, int U = N == 4 ? 16 : 2>
__device__ __forceinline__ float merge_row(const float* part_out, const float* part_lse,
                                           int s0, int ns, int R, int row, int lane, const float* sink,
                                           int head, float (&acc)[N], int k0 = 0) {
  constexpr int K = N / 4;
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  float lse_tot;
  if (ns <= 4) {
    // up to 4 splits (the common case): every load first, in one round trip to memory
    float ls[4];
    float4 v[4][K];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      ls[s] = -INFINITY;
      if (s < ns) {
        ls[s] = part_lse[(int64_t)(s0 + s) * R + row];
        const float4* src = reinterpret_cast<const float4*>(part_out + ((int64_t)(s0 + s) * R + row) * 512);
#pragma unroll
        for (int k = 0; k < K; ++k) v[s][k] = src[(k0 + k) * 32 + lane];
      }
    }
    bool any = false;
#pragma unroll
    for (int s = 0; s < 4; ++s) any |= ls[s] != -INFINITY;
    if (!any) return -INFINITY;
    const float mx = fmaxf(fmaxf(ls[0], ls[1]), fmaxf(ls[2], ls[3]));
    float tot = 0.f;
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (s < ns) tot += expf(ls[s] - mx);
    lse_tot = mx + logf(tot);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s >= ns || ls[s] == -INFINITY) continue;
      const float w = expf(ls[s] - lse_tot);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        acc[4 * k + 0] += w * v[s][k].x;
        acc[4 * k + 1] += w * v[s][k].y;
        acc[4 * k + 2] += w * v[s][k].z;
        acc[4 * k + 3] += w * v[s][k].w;
      }
    }
  } else {
    float mx = -INFINITY;
    bool any = false;
    for (int s = lane; s < ns; s += 32) {
      const float l = part_lse[(int64_t)(s0 + s) * R + row];
      mx = fmaxf(mx, l);
      any |= l != -INFINITY;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (!__any_sync(0xffffffffu, any)) return -INFINITY;
    float tot = 0.f;
    for (int s = lane; s < ns; s += 32) tot += expf(part_lse[(int64_t)(s0 + s) * R + row] - mx);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    lse_tot = mx + logf(tot);
    // Weights 32 splits at a time, a lane each; then the splits in order, U of them loaded at once: each element's sum
    // is the same as one by one, without a round trip to memory for each split.
    for (int base = 0; base < ns; base += 32) {
      const float ls = base + lane < ns ? part_lse[(int64_t)(s0 + base + lane) * R + row] : -INFINITY;
      const float wl = expf(ls - lse_tot);
      const unsigned on = __ballot_sync(0xffffffffu, ls != -INFINITY);
      for (int u = 0; u < 32 && base + u < ns; u += U) {
        float4 v[U][K];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (!((on >> (u + i)) & 1u)) continue;
          const float4* src = reinterpret_cast<const float4*>(part_out + ((int64_t)(s0 + base + u + i) * R + row) * 512);
#pragma unroll
          for (int k = 0; k < K; ++k) v[i][k] = src[(k0 + k) * 32 + lane];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float w = __shfl_sync(0xffffffffu, wl, u + i);
          if (!((on >> (u + i)) & 1u)) continue;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            acc[4 * k + 0] += w * v[i][k].x;
            acc[4 * k + 1] += w * v[i][k].y;
            acc[4 * k + 2] += w * v[i][k].z;
            acc[4 * k + 3] += w * v[i][k].w;
          }
        }
      }
    }
  }
  float f = 1.f;
  if (sink != nullptr) f = 1.f / (1.f + expf(sink[head] - lse_tot));
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] *= f;
  return lse_tot;
}

// Round a merged row (or quarter k0 of it) to bf16 and store it (dst = the row's 512 elements), rounding acc in place.
template <int N>
__device__ __forceinline__ void store_row_bf16(uint16_t* dst, int lane, float (&acc)[N], int k0 = 0) {
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    const uint32_t lo = f32x2_to_bf16x2(acc[4 * k], acc[4 * k + 1]);
    const uint32_t hi = f32x2_to_bf16x2(acc[4 * k + 2], acc[4 * k + 3]);
    *reinterpret_cast<uint2*>(dst + ((k0 + k) * 32 + lane) * 4) = make_uint2(lo, hi);
    acc[4 * k] = __uint_as_float(lo << 16);
    acc[4 * k + 1] = __uint_as_float(lo & 0xFFFF0000u);
    acc[4 * k + 2] = __uint_as_float(hi << 16);
    acc[4 * k + 3] = __uint_as_float(hi & 0xFFFF0000u);
  }
}

}  // namespace mla
