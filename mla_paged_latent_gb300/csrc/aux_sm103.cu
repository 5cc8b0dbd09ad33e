// Split combine, KV-row write and page gather kernels for sm_103a.
#include <cstdint>
#include <cuda_runtime.h>

#include "combine_row.cuh"
#include "kv_row.cuh"
#include "mla_kernels.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

// ----------------------------------------------------------------------------- combine
// One warp per query row of a request that the plan split into >= 2 pieces (the merge
// itself is merge_row in combine_row.cuh), or with few rows WARPS = 4 of them, a quarter of the row each.
template <int WARPS>
__global__ void __launch_bounds__(128) combine_kernel(const float* part_out, const float* part_lse,
                                                      const int32_t* num_splits, int R, int heads, const float* sink,
                                                      uint16_t* out, float* lse, const float* part_max,
                                                      float* max_logits) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y;
  const int s0 = num_splits[b];
  const int ns = num_splits[b + 1] - s0;
  if (ns < 2) return;
  const int wi = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int row = wi / WARPS, k0 = wi % WARPS;
  if (row >= R) return;
  const int lane = threadIdx.x & 31;
  const int64_t orow = (int64_t)b * R + row;
  float acc[16 / WARPS];
  const float lse_tot = merge_row(part_out, part_lse, s0, ns, R, row, lane, sink, row % heads, acc, k0);
  store_row_bf16(out + orow * 512, lane, acc, k0);
  if (k0 != 0) return;
  if (lane == 0) lse[orow] = lse_tot;
  if (max_logits != nullptr) {  // the largest scaled score: the largest over the splits
    float m = -INFINITY;
    for (int s = lane; s < ns; s += 32) m = fmaxf(m, part_max[(int64_t)(s0 + s) * R + row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) max_logits[orow] = m;
  }
}

// One warp per query row: the merged (split) or decode-written (unsplit) row, with the
// inverse RoPE applied to elements [rope0, rope0 + 64): pair i = (u, v) -> (u c + v s,
// v c - u s), (c, s) = freqs[pos, 2i], freqs[pos, 2i + 1] ("MLA" API page of HALOps,
// mla_output_proj: the split-KV partials merged by LSE, then the RoPE of O undone). Written
// back to out.
__global__ void __launch_bounds__(256) combine_inv_rope_kernel(
    const float* part_out, const float* part_lse, const int32_t* num_splits,
    int R, int sq, int heads, const float* sink, const int32_t* positions,
    const float* freqs, int max_pos, int rope0, uint16_t* out, float* lse) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= R) return;
  const int lane = threadIdx.x & 31;
  const int64_t orow = (int64_t)b * R + row;
  const int s0 = num_splits[b];
  const int ns = num_splits[b + 1] - s0;
  const int pos = positions[b * sq + row / heads];
  float acc[16];
  if (ns >= 2 && part_out != nullptr) {  // no partials given: every row is taken as written
    const float lse_tot = merge_row(part_out, part_lse, s0, ns, R, row, lane, sink, row % heads, acc);
    store_row_bf16(out + orow * 512, lane, acc);  // acc now holds the bf16 values
    if (lane == 0) lse[orow] = lse_tot;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint2 v = *reinterpret_cast<const uint2*>(out + orow * 512 + (k * 32 + lane) * 4);
      acc[4 * k] = __uint_as_float(v.x << 16);
      acc[4 * k + 1] = __uint_as_float(v.x & 0xFFFF0000u);
      acc[4 * k + 2] = __uint_as_float(v.y << 16);
      acc[4 * k + 3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
  }
  if (pos < 0 || pos >= max_pos) return;  // no table row: left as merged
  const float* f = freqs + (int64_t)pos * 64;
  // lane holds elements d = 4 (32 k + lane) .. +3, i.e. pairs (d, d + 1) and (d + 2, d + 3)
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int d = (k * 32 + lane) * 4;
    if (d < rope0 || d >= rope0 + 64) continue;
    const int i = (d - rope0) >> 1;
    float y[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float c = f[2 * (i + h)], sn = f[2 * (i + h) + 1];
      const float u = acc[4 * k + 2 * h], v = acc[4 * k + 2 * h + 1];
      y[2 * h] = u * c + v * sn;
      y[2 * h + 1] = v * c - u * sn;
    }
    *reinterpret_cast<uint2*>(out + orow * 512 + d) = make_uint2(f32x2_to_bf16x2(y[0], y[1]), f32x2_to_bf16x2(y[2], y[3]));
  }
}

// ----------------------------------------------------------------------------- window runs
// One warp per token: compress its window (kv_indices[t, 0 .. len), len = topk_lengths[t]
// clamped to [0, topk], or topk) into at most two runs of consecutive cache slots ("MLA" API
// page of HALOps, mla_attention_plan). A run continues while the next slot is the previous
// one plus kv_run_step and lies on the same page; a window of more than two runs is cut to
// its first row. Each run is stored from its lowest slot upwards (attention does not depend
// on the order of its rows): row g < len0 is slot slot0 + g, row g >= len0 slot1 + g - len0.
// The lanes read 32 window entries at a time and find the run breaks with one ballot.
__global__ void __launch_bounds__(128) swa_plan_kernel(const int32_t* idx, const int32_t* lens, int T, int topk,
                                                       int log2_ps, int step, int4* runs) {
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= T) return;
  int len = lens ? lens[t] : topk;
  len = len < 0 ? 0 : (len > topk ? topk : len);
  if (len == 0) {
    if (lane == 0) runs[t] = make_int4(0, 0, 0, 0);
    return;
  }
  const int32_t* w = idx + (int64_t)t * topk;
  const int first = w[0];
  int nb = 0, b1 = len, s1 = 0;  // breaks found; row and slot of the first break
  int carry = first;
  for (int base = 0; base < len && nb < 2; base += 32) {
    const int g = base + lane;
    const bool valid = g < len;
    const int cur = valid ? w[g] : 0;
    int prev = __shfl_up_sync(0xffffffffu, cur, 1);
    if (lane == 0) prev = carry;
    const bool brk = valid && g > 0 && (cur != prev + step || (cur >> log2_ps) != (prev >> log2_ps));
    unsigned m = __ballot_sync(0xffffffffu, brk);
    while (m != 0u && nb < 2) {
      const int l = __ffs(m) - 1;
      const int v = __shfl_sync(0xffffffffu, cur, l);
      if (nb == 0) {
        b1 = base + l;
        s1 = v;
      }
      ++nb;
      m &= m - 1u;
    }
    carry = __shfl_sync(0xffffffffu, cur, 31);
  }
  if (lane != 0) return;
  if (nb >= 2) {
    runs[t] = make_int4(first, 1, first, 1);
    return;
  }
  const int c0 = b1;  // len when the window is one run
  const int lo0 = step > 0 ? first : first - (c0 - 1);
  const int lo1 = nb == 1 ? (step > 0 ? s1 : s1 - (len - b1 - 1)) : lo0 + c0;
  runs[t] = make_int4(lo0, c0, lo1, len);
}

// ----------------------------------------------------------------------------- kv write
// One warp per new row, already normalised. A kernel a layout, the page by a shift: bound by a row's instructions
// (65000 rows of layouts 0, 1, 2: 23.1, 22.5, 23.2 us, 4.7 to 6.5 TB/s; with the layout as an argument and a division
// 27.2, 29.7, 29.9).
template <int LAYOUT>
__global__ void __launch_bounds__(128) kv_write_kernel(const uint16_t* rows, const int32_t* slots, int n, uint8_t* kv,
                                                       int64_t num_pages, int page_size, int64_t page_bytes,
                                                       uint32_t* status) {
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= n) return;
  const int slot = slots[r];
  if (slot < 0) return;
  const int64_t page = slot >> (31 - __clz(page_size));  // (a power of two)
  if (page >= num_pages) {  // reported, not written
    if (lane == 0 && status != nullptr) atomicOr(status, 4u);
    return;
  }
  write_row(rows + (int64_t)r * row_width(LAYOUT), lane, kv, LAYOUT, page, slot & (page_size - 1), page_size,
            page_bytes);
}

// The same for 4-bit rows. Bound by the length of a row's chain (one row a warp, as many warps as fit) and by its
// instructions. So the row is loaded beside its slot and not after it, and the largest magnitude of a group and its
// NaNs are found at once, on bf16 pairs taken as integers: 65000 rows of 448 + 64 20 us against 29 with neither; 16.9 us
// (5.4 TB/s) since the row's arithmetic is in 32 bits.
template <int LAYOUT>
__global__ void __launch_bounds__(256) kv_write_fp4_kernel(const uint16_t* rows, const int32_t* slots, int n,
                                                           uint8_t* kv, int64_t num_pages, int page_size,
                                                           int64_t page_bytes, uint32_t* status) {
  pdl_trigger();
  pdl_wait();
  constexpr int kNope = row_nope(LAYOUT), kRowBytes = row_stored_bytes(LAYOUT);
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= n) return;
  const uint4* x = reinterpret_cast<const uint4*>(rows + (int64_t)r * row_width(LAYOUT));
  const uint4 x0 = x[2 * lane], x1 = x[2 * lane + 1], pe = x[kNope / 8 + (lane & 7)];
  const int slot = slots[r];
  if (slot < 0) return;
  const int page = slot >> (31 - __clz(page_size));  // (a power of two)
  const int off = slot & (page_size - 1);
  if (page >= num_pages) {  // reported, not written
    if (lane == 0 && status != nullptr) atomicOr(status, 4u);
    return;
  }
  uint8_t* const pg = kv + page * page_bytes;
  write_row_fp4(x0, x1, pe, lane, kNope, pg + (int64_t)off * kRowBytes,
                pg + (int64_t)page_size * kRowBytes + (int64_t)off * kFp4ScaleSlot);
}

// One warp per raw row: RMSNorm of the 512 latent elements and RoPE of the 64 RoPE
// elements in fp32 ("MLA" API page of HALOps, mla_attention: its normalise-and-rotate
// step before the cache write, kv_norm_weight / kv_eps / positions / freqs_real), the row
// rounded to bf16 in shared memory (norm_rope_row), then written as write_row writes it.
__global__ void __launch_bounds__(128) kv_write_norm_rope_kernel(
    const uint16_t* raw, const int32_t* slots, const int32_t* positions,
    const uint16_t* w, float eps, const float* freqs, int max_pos, int n,
    uint8_t* kv, int layout, int64_t num_pages, int page_size, int64_t page_bytes, uint32_t* status) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) uint16_t srow[4][576];
  const int wi = threadIdx.x >> 5;
  const int r = blockIdx.x * 4 + wi;
  const int lane = threadIdx.x & 31;
  if (r >= n) return;
  const int64_t slot = slots[r];
  if (slot < 0) return;
  const int64_t page = slot / page_size;
  const int pos = positions[r];
  const uint32_t bad = (page >= num_pages ? 4u : 0u) | (pos < 0 || pos >= max_pos ? 8u : 0u);
  if (bad != 0u) {  // reported, not written
    if (lane == 0 && status != nullptr) atomicOr(status, bad);
    return;
  }
  const int row_elems = row_width(layout);
  const uint16_t* x = raw + (int64_t)r * row_elems;
  const float* f = freqs + (int64_t)pos * 64;
  norm_rope_row(x, w, eps, f, row_elems, lane, srow[wi]);
  write_any_row(srow[wi], lane, kv, layout, page, static_cast<int>(slot % page_size), page_size, page_bytes);
}

// ----------------------------------------------------------------------------- gather
__global__ void __launch_bounds__(128) kv_gather_kernel(const uint8_t* kv, int layout, int64_t num_pages,
                                                        int page_size, int64_t page_bytes, const int32_t* bt_row,
                                                        int max_pages, int length, float* out) {
  pdl_trigger();
  pdl_wait();
  const int j = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (j >= length) return;
  const int dqk = row_width(layout);
  float* o = out + (int64_t)j * dqk;
  const int pi = j / page_size;
  const int64_t page = pi < max_pages ? bt_row[pi] : -1;
  if (page < 0 || page >= num_pages) {
    for (int d = lane; d < dqk; d += 32) o[d] = __uint_as_float(0x7FC00000u);
    return;
  }
  const int off = j % page_size;
  if (layout == 0) {
    const uint16_t* src = reinterpret_cast<const uint16_t*>(kv + page * page_bytes + (int64_t)off * 1152);
    for (int d = lane; d < 576; d += 32) o[d] = bf16_to_f32(src[d]);
    return;
  }
  const int nope = row_nope(layout);
  const int row_bytes = row_stored_bytes(layout);
  const uint8_t* src = kv + page * page_bytes + (int64_t)off * row_bytes;
  const uint8_t* sc = kv + page * page_bytes + (int64_t)page_size * row_bytes + (int64_t)off * row_scale_slot(layout);
  if (layout >= 3) {
    for (int i = lane; i < nope / 8; i += 32) {
      uint32_t o4[4];
      fp4x8_to_bf16(reinterpret_cast<const uint32_t*>(src)[i], fp4_scale(sc[i >> 2]), o4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[8 * i + 2 * k] = bf16_to_f32(o4[k] & 0xFFFFu);
        o[8 * i + 2 * k + 1] = bf16_to_f32(o4[k] >> 16);
      }
    }
    const uint16_t* pe = reinterpret_cast<const uint16_t*>(src + nope / 2);
    for (int d = lane; d < 64; d += 32) o[nope + d] = bf16_to_f32(pe[d]);
    return;
  }
  for (int d = 2 * lane; d < nope; d += 64) {
    const uint32_t two = *reinterpret_cast<const uint16_t*>(src + d);
    const float2 v = e4m3x2_to_f32x2(two);
    const float s = ue8m0_to_f32(sc[d >> 6]);
    o[d] = v.x * s;
    o[d + 1] = v.y * s;
  }
  const uint16_t* rope = reinterpret_cast<const uint16_t*>(src + nope);
  for (int d = lane; d < 64; d += 32) o[nope + d] = bf16_to_f32(rope[d]);
}

}  // namespace

cudaError_t launch_combine(const float* part_out, const float* part_lse, const int32_t* num_splits, int batch,
                           int rows_per_req, int heads, const float* sink, uint16_t* out, float* lse,
                           const float* part_max, float* max_logits, cudaStream_t stream) {
  if (batch <= 0 || rows_per_req <= 0) return cudaSuccess;
  // Blocks of 128 threads: 94 registers a thread with a warp a row (five blocks an SM, against two of 256 threads), 114
  // with four warps a row (four). Four warps a row where rows are few: a few requests split many ways are bound by the
  // loads that a warp keeps in flight. Measured, us a launch, partials of 2 / 4 / 8 / 16 / 76 splits out of L2 and DRAM in
  // turn, four warps a row against one:
  //   128 rows  1.5 / 1.7 / 2.8 / 3.0 / 14.1   1.6 / 1.8 / 3.1 / 4.3 / 29.5
  //   384       1.6 / 2.0 / 3.2 / 4.9 / 16.3   1.7 / 2.1 / 3.3 / 8.0 / 30.3
  //   512       1.7 / 1.9 / 3.4 / 5.8 / 17.8   1.9 / 2.2 / 3.9 / 8.6 / 31.1
  //   640       2.2 / 2.5 / 5.1 / 8.8 / 29.9   2.1 / 2.5 / 4.7 / 9.0 / 32.7
  const bool few = static_cast<int64_t>(rows_per_req) * batch <= 512;
  const dim3 grid(few ? rows_per_req : (rows_per_req + 3) / 4, batch);
  return launch_pdl(few ? combine_kernel<4> : combine_kernel<1>, grid, dim3(128), 0, stream, part_out, part_lse,
                    num_splits, rows_per_req, heads, sink, out, lse, part_max, max_logits);
}

cudaError_t launch_swa_plan(const int32_t* kv_indices, const int32_t* topk_lengths, int num_tokens, int topk,
                            int page_size, int kv_run_step, int32_t* runs, cudaStream_t stream) {
  int lg = 0;
  while ((1 << lg) < page_size) ++lg;
  return launch_pdl(swa_plan_kernel, dim3((num_tokens + 3) / 4), dim3(128), 0, stream, kv_indices, topk_lengths,
                    num_tokens, topk, lg, kv_run_step, reinterpret_cast<int4*>(runs));
}

cudaError_t launch_combine_inv_rope(const float* part_out, const float* part_lse, const int32_t* num_splits, int batch,
                                    int sq, int heads, const float* sink, const int32_t* positions, const float* freqs,
                                    int max_pos, int rope0, uint16_t* out, float* lse, cudaStream_t stream) {
  const int R = sq * heads;
  dim3 grid((R + 7) / 8, batch);
  return launch_pdl(combine_inv_rope_kernel, grid, dim3(256), 0, stream, part_out, part_lse, num_splits, R, sq, heads,
                    sink, positions, freqs, max_pos, rope0, out, lse);
}

cudaError_t launch_kv_write(const uint16_t* rows, const int32_t* slots, int n, uint8_t* kv, int layout,
                            int64_t num_pages, int page_size, int64_t page_bytes, uint32_t* status,
                            cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  if (layout >= 3)
    return launch_pdl(layout == 3 ? kv_write_fp4_kernel<3> : kv_write_fp4_kernel<4>, dim3((n + 7) / 8), dim3(256), 0,
                      stream, rows, slots, n, kv, num_pages, page_size, page_bytes, status);
  return launch_pdl(layout == 0   ? kv_write_kernel<0>
                    : layout == 1 ? kv_write_kernel<1>
                                  : kv_write_kernel<2>,
                    dim3((n + 3) / 4), dim3(128), 0, stream, rows, slots, n, kv, num_pages, page_size, page_bytes, status);
}

cudaError_t launch_kv_write_norm_rope(const uint16_t* raw, const int32_t* slots, const int32_t* positions,
                                     const uint16_t* norm_weight, float eps, const float* freqs, int max_pos, int n,
                                     uint8_t* kv, int layout, int64_t num_pages, int page_size, int64_t page_bytes,
                                     uint32_t* status, cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  return launch_pdl(kv_write_norm_rope_kernel, dim3((n + 3) / 4), dim3(128), 0, stream, raw, slots, positions,
                    norm_weight, eps, freqs, max_pos, n, kv, layout, num_pages, page_size, page_bytes, status);
}

cudaError_t launch_kv_gather(const uint8_t* kv, int layout, int64_t num_pages, int page_size, int64_t page_bytes,
                             const int32_t* bt_row, int max_pages, int length, float* out, cudaStream_t stream) {
  if (length <= 0) return cudaSuccess;
  return launch_pdl(kv_gather_kernel, dim3((length + 3) / 4), dim3(128), 0, stream, kv, layout, num_pages, page_size,
                    page_bytes, bt_row, max_pages, length, out);
}

}  // namespace mla
