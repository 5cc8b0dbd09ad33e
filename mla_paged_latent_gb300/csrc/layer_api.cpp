// C ABI of the steps of a chunk of new tokens around the cache: attention in its per-head form and the matrix product
// with an epilogue. Argument checks, tensor maps and launches; include/mla_decode.h says what every argument means.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>

#include "api_common.h"
#include "mla_decode.h"
#include "mla_kernels.h"

namespace {

using mla::aligned_to;
using mla::ByteRange;
using mla::bytes_at;
using mla::cuda_fail;
using mla::fail;
using mla::overlap;

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// A map of bf16 rows: `cols` elements, `rows` of them `stride` elements apart, moved in boxes of box_cols x box_rows.
int rows_map(const char* what, CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t stride, int box_cols,
             int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  return mla::encode_bf16_map(what, map, base, 2, dims, strides, box);
}

// Where the parts of a chunk's workspace begin (bytes).
struct ChunkSpace {
  size_t rows, kv, value_wide, any_wide, part_out, part_lse, end;
};
ChunkSpace chunk_space(int64_t kv_rows, int64_t heads, int64_t group, int64_t slots) {
  ChunkSpace s;
  const size_t n = static_cast<size_t>(kv_rows < 128 ? 128 : kv_rows);
  s.rows = MLA_WORKSPACE_HEADER;
  s.kv = s.rows + align256(n * 1152);
  s.value_wide = s.kv + n * static_cast<size_t>(group) * 512;
  s.any_wide = s.value_wide + align256(n / 32 * static_cast<size_t>(group));
  s.part_out = s.any_wide + align256(static_cast<size_t>((heads + group - 1) / group) * 4);
  s.part_lse = s.part_out + static_cast<size_t>(slots) * 128 * 4;
  s.end = s.part_lse + static_cast<size_t>(slots) * 4;
  return s;
}

// Sections of the schedule (32-bit words), each a multiple of four.
struct ChunkSections {
  int64_t pair_items, items, merges, end;  // (the first begins at 0)
};
ChunkSections chunk_sections(const mla_chunk_info& i) {
  auto four = [](int64_t x) { return (x + 3) & ~int64_t(3); };
  ChunkSections s;
  s.pair_items = 4 * static_cast<int64_t>(i.kv_rows / 128);
  s.items = s.pair_items + four(i.pairs + 1);
  s.merges = s.items + 12 * static_cast<int64_t>(i.items);
  s.end = s.merges + 8 * static_cast<int64_t>(i.merges);
  return s;
}

}  // namespace

extern "C" {

int mla_chunk_plan(const int32_t* q_lens, const int32_t* kv_lens, int32_t batch, int32_t num_heads, int32_t causal,
                   size_t kv_budget, int32_t num_sms, int32_t* sched, int64_t sched_capacity, mla_chunk_info* info) {
  if (!q_lens || !kv_lens || !info) return fail(MLA_ERR_INVALID_ARG, "mla_chunk_plan: NULL argument");
  if (batch < 1 || num_heads < 1 || num_sms < 2)
    return fail(MLA_ERR_INVALID_ARG, "mla_chunk_plan: batch=%d heads=%d num_sms=%d out of range", batch, num_heads, num_sms);
  int64_t tokens = 0, rows = 0, tiles = 0;
  for (int b = 0; b < batch; ++b) {
    if (q_lens[b] < 0 || kv_lens[b] < 0)
      return fail(MLA_ERR_INVALID_ARG, "mla_chunk_plan: lengths of request %d are %d and %d", b, q_lens[b], kv_lens[b]);
    tokens += q_lens[b];
    tiles += (static_cast<int64_t>(q_lens[b]) + 511) / 512;
    if (q_lens[b] > 0) rows += (static_cast<int64_t>(kv_lens[b]) + 127) / 128 * 128;
  }
  if (num_heads > 4096 || tokens * num_heads >= (1ll << 31) - 512 || rows >= (1ll << 31) - 512)
    return fail(MLA_ERR_UNSUPPORTED, "mla_chunk_plan: %lld tokens of %d heads over %lld rows are too many",
                static_cast<long long>(tokens), num_heads, static_cast<long long>(rows));
  // heads whose K and V are held at once: as many as the budget takes, in groups of about the same size
  const int64_t per_head = (rows < 128 ? 128 : rows) * 512;
  int64_t group = static_cast<int64_t>(kv_budget / static_cast<size_t>(per_head));
  group = group < 1 ? 1 : group > num_heads ? num_heads : group;
  const int64_t groups = (num_heads + group - 1) / group;
  group = (num_heads + groups - 1) / groups;
  if (tiles * group > (1ll << 27))  // (words of the schedule are found by 32-bit indices, 12 of them a unit)
    return fail(MLA_ERR_UNSUPPORTED, "mla_chunk_plan: %lld query tiles of %lld heads at once are too many units",
                static_cast<long long>(tiles), static_cast<long long>(group));
  try {
    const mla::ChunkPlan p = mla::make_chunk_plan(q_lens, kv_lens, batch, num_heads, causal != 0, static_cast<int>(group), num_sms);
    std::memset(info, 0, sizeof *info);
    info->batch = batch;
    info->heads = num_heads;
    info->causal = causal ? 1 : 0;
    info->tokens = static_cast<int32_t>(tokens);
    info->kv_rows = static_cast<int32_t>(rows);
    info->group = static_cast<int32_t>(group);
    info->pairs = static_cast<int32_t>(p.pair_items.size()) - 1;
    info->items = static_cast<int32_t>(p.items.size() / 12);
    info->merges = static_cast<int32_t>(p.merges.size() / 8);
    info->slots = p.slots;
    const ChunkSections s = chunk_sections(*info);
    info->sched_words = s.end;
    info->workspace_bytes = chunk_space(rows, num_heads, group, p.slots).end;
    if (sched == nullptr) return MLA_OK;
    if (sched_capacity < s.end)
      return fail(MLA_ERR_CAPACITY, "mla_chunk_plan: sched needs %lld words, capacity %lld", static_cast<long long>(s.end),
                  static_cast<long long>(sched_capacity));
    std::memset(sched, 0, static_cast<size_t>(s.end) * 4);
    auto put = [&](int64_t at, const std::vector<int32_t>& v) {
      if (!v.empty()) std::memcpy(sched + at, v.data(), v.size() * 4);
    };
    put(0, p.kv_tiles);
    put(s.pair_items, p.pair_items);
    put(s.items, p.items);
    put(s.merges, p.merges);
  } catch (const std::bad_alloc&) {
    return fail(MLA_ERR_UNSUPPORTED, "mla_chunk_plan: out of host memory");
  }
  return MLA_OK;
}

int mla_chunk_attention(const void* q, const void* kv_cache, mla_kv_layout layout, int64_t num_pages, int32_t page_size,
                        const int32_t* block_table, int32_t max_pages, const void* w_kv, float sm_scale,
                        const mla_chunk_info* info, const int32_t* sched, void* workspace, size_t workspace_bytes, void* out,
                        float* lse, void* stream) {
  if (!info) return fail(MLA_ERR_INVALID_ARG, "mla_chunk_attention: NULL plan");
  const mla_chunk_info& I = *info;
  if (I.batch < 1 || I.heads < 1 || I.heads > 4096 || I.tokens < 0 || I.kv_rows < 0 || I.kv_rows % 128 != 0 || I.group < 1 ||
      I.group > I.heads || I.pairs < 0 || I.items < I.pairs || I.merges < 0 || I.slots < I.merges ||
      static_cast<int64_t>(I.tokens) * I.heads >= (1ll << 31) - 512 || I.sched_words != chunk_sections(I).end)
    return fail(MLA_ERR_INVALID_ARG, "mla_chunk_attention: the plan is not one that mla_chunk_plan made");
  if (I.tokens == 0) return MLA_OK;
  if (!q || !kv_cache || !block_table || !w_kv || !sched || !workspace || !out)
    return fail(MLA_ERR_INVALID_ARG, "mla_chunk_attention: NULL pointer argument");
  int64_t row_bytes, page_bytes;
  int dqk;
  if (mla::layout_geometry(layout, page_size, &row_bytes, &page_bytes, &dqk) != 0)
    return fail(MLA_ERR_INVALID_ARG, "mla_chunk_attention: unknown layout %d", static_cast<int>(layout));
  if (dqk != 576)
    return fail(MLA_ERR_UNSUPPORTED, "mla_chunk_attention: layout %d has 512-wide rows, which are keys and values themselves",
                static_cast<int>(layout));
  if (page_size < 8 || (page_size & (page_size - 1)) != 0)
    return fail(MLA_ERR_UNSUPPORTED, "mla_chunk_attention: page_size %d must be a power of two >= 8", page_size);
  if (num_pages < 1 || max_pages < 1)
    return fail(MLA_ERR_INVALID_ARG, "mla_chunk_attention: num_pages and max_pages must be >= 1");
  if (!(sm_scale > 0.f) || !(sm_scale < 1e30f))
    return fail(MLA_ERR_INVALID_ARG, "mla_chunk_attention: sm_scale must be a positive finite number");
  if (!aligned_to(q, 16) || !aligned_to(kv_cache, 16) || !aligned_to(w_kv, 16) || !aligned_to(sched, 16) ||
      !aligned_to(out, 32) || !aligned_to(lse, 4) || !aligned_to(block_table, 4))
    return fail(MLA_ERR_INVALID_ARG, "mla_chunk_attention: q, kv_cache, w_kv and sched must be 16-byte and out 32-byte aligned");
  if (!aligned_to(workspace, 256)) return fail(MLA_ERR_INVALID_ARG, "mla_chunk_attention: workspace must be 256-byte aligned");
  const ChunkSpace space = chunk_space(I.kv_rows, I.heads, I.group, I.slots);
  if (workspace_bytes < space.end)
    return fail(MLA_ERR_WORKSPACE_TOO_SMALL, "mla_chunk_attention: workspace %zu bytes < %zu needed", workspace_bytes, space.end);
  const int64_t T = I.tokens, N = I.heads;
  const ByteRange written[3] = {bytes_at(out, T * N * 256), bytes_at(lse, lse ? T * N * 4 : 0), bytes_at(workspace, space.end)};
  const ByteRange read[5] = {bytes_at(q, T * N * 384), bytes_at(kv_cache, num_pages * page_bytes), bytes_at(w_kv, N * 256 * 1024),
                             bytes_at(sched, I.sched_words * 4), bytes_at(block_table, 4ll * I.batch * max_pages)};
  for (int i = 0; i < 3; ++i) {
    for (const ByteRange& r : read)
      if (overlap(written[i], r)) return fail(MLA_ERR_INVALID_ARG, "mla_chunk_attention: out, lse or workspace overlaps an input");
    for (int k = 0; k < i; ++k)
      if (overlap(written[i], written[k])) return fail(MLA_ERR_INVALID_ARG, "mla_chunk_attention: out, lse and workspace overlap");
  }

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const ChunkSections at = chunk_sections(I);
  mla::ChunkParams p;
  std::memset(&p, 0, sizeof p);
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.block_table = block_table;
  p.rows = reinterpret_cast<uint16_t*>(ws + space.rows);
  p.kv_tiles = sched;
  p.pair_items = sched + at.pair_items;
  p.items = sched + at.items;
  p.merges = sched + at.merges;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.value_wide = ws + space.value_wide;
  p.part_out = reinterpret_cast<float*>(ws + space.part_out);
  p.part_lse = reinterpret_cast<float*>(ws + space.part_lse);
  p.status = reinterpret_cast<unsigned int*>(ws);
  p.num_pages = num_pages;
  p.page_bytes = page_bytes;
  p.page_size = page_size;
  while ((1 << p.log2_ps) < page_size) ++p.log2_ps;
  p.max_pages = max_pages;
  p.kv_rows = I.kv_rows;
  p.tokens = I.tokens;
  p.heads = I.heads;
  p.causal = I.causal;
  p.scale_log2 = sm_scale * 1.4426950408889634f;

  const void* kv = ws + space.kv;
  const int64_t rows = I.kv_rows < 128 ? 128 : I.kv_rows, kv_cols = static_cast<int64_t>(I.group) * 256;
  CUtensorMap q_map, kv_map, rope_map, x_map, w_map, y_map;
  {
    const cuuint64_t dims[3] = {192, static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[2] = {384, static_cast<cuuint64_t>(N) * 384};
    const cuuint32_t box[3] = {64, 1, 128};
    if (int rc = mla::encode_bf16_map("mla_chunk_attention: q", &q_map, q, 3, dims, strides, box)) return rc;
  }
  if (int rc = rows_map("mla_chunk_attention: K and V", &kv_map, kv, kv_cols, rows, kv_cols, 64, 64)) return rc;
  if (int rc = rows_map("mla_chunk_attention: RoPE rows", &rope_map, p.rows, 576, rows, 576, 64, 64)) return rc;
  if (int rc = rows_map("mla_chunk_attention: latent rows", &x_map, p.rows, 512, rows, 576, 64, 128)) return rc;
  if (int rc = rows_map("mla_chunk_attention: w_kv", &w_map, w_kv, 512, N * 256, 512, 64, 128)) return rc;
  if (int rc = rows_map("mla_chunk_attention: K and V out", &y_map, kv, kv_cols, rows, kv_cols, 64, 32)) return rc;
  int num_sms = 0;
  if (int rc = mla::current_sm_count(&num_sms)) return rc;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  int32_t* any_wide = reinterpret_cast<int32_t*>(ws + space.any_wide);  // of each group of heads
  if (I.kv_rows > 0) {
    p.any_wide = any_wide;
    p.group_heads = I.group;
    e = mla::launch_chunk_rows(static_cast<int>(layout), p, s);
    if (e != cudaSuccess) return cuda_fail(e, "mla_chunk_attention: rows launch");
  }
  for (int head0 = 0; head0 < I.heads; head0 += I.group, ++any_wide) {
    p.head0 = head0;
    p.any_wide = any_wide;
    p.group_heads = I.heads - head0 < I.group ? I.heads - head0 : I.group;
    if (I.kv_rows > 0) {
      mla::GemmParams g;
      std::memset(&g, 0, sizeof g);
      g.status = p.status;
      g.value_wide = ws + space.value_wide;
      g.value_wide_stride = I.kv_rows / 32;
      g.any_wide = any_wide;
      g.rows = I.kv_rows;
      g.cols = p.group_heads * 256;
      g.k_blocks = 8;
      g.m_tiles = (g.rows + 255) / 256;
      g.n_tiles = p.group_heads;
      g.band = 8;
      g.tile_cols = 256;
      g.w_row0 = head0 * 256;
      const int64_t tiles = static_cast<int64_t>(g.m_tiles) * g.n_tiles;
      e = mla::launch_gemm_pair(g, x_map, w_map, y_map, static_cast<int>(tiles < num_sms / 2 ? tiles : num_sms / 2), s);
      if (e != cudaSuccess) return cuda_fail(e, "mla_chunk_attention: up-projection launch");
    }
    e = mla::launch_chunk_attention(p, q_map, kv_map, rope_map, I.pairs, s);
    if (e != cudaSuccess) return cuda_fail(e, "mla_chunk_attention: attention launch");
    if (I.merges > 0) {
      e = mla::launch_chunk_merge(p, I.merges, s);
      if (e != cudaSuccess) return cuda_fail(e, "mla_chunk_attention: merge launch");
    }
  }
  return MLA_OK;
}

int mla_linear(const void* x, int64_t x_stride, const void* weight, const void* bias, const void* residual,
               int64_t residual_stride, int32_t activation, int32_t rows, int32_t inner, int32_t outer, void* out,
               int64_t out_stride, uint32_t* status, void* stream) {
  if (rows < 0 || inner < 1 || outer < 1)
    return fail(MLA_ERR_INVALID_ARG, "mla_linear: rows=%d inner=%d outer=%d out of range", rows, inner, outer);
  if (rows == 0) return MLA_OK;
  if (!x || !weight || !out) return fail(MLA_ERR_INVALID_ARG, "mla_linear: NULL pointer argument");
  if (inner % 8 != 0 || outer % 8 != 0)
    return fail(MLA_ERR_UNSUPPORTED, "mla_linear: inner %d and outer %d must be multiples of 8", inner, outer);
  if (activation < MLA_ACT_NONE || activation > MLA_ACT_GELU)
    return fail(MLA_ERR_INVALID_ARG, "mla_linear: unknown activation %d", activation);
  if (inner > (1 << 30) || outer > (1 << 30) || rows > (1 << 30))
    return fail(MLA_ERR_UNSUPPORTED, "mla_linear: a size above 2^30");
  if (rows == 1) {  // the stride of one row is not read
    x_stride = inner;
    residual_stride = out_stride = outer;
  }
  if (!residual) residual_stride = outer;
  const int64_t strides[3] = {x_stride, residual_stride, out_stride}, widths[3] = {inner, outer, outer};
  for (int i = 0; i < 3; ++i)
    if (strides[i] < widths[i] || strides[i] % 8 != 0 || strides[i] > (1ll << 46) / rows)  // (past any memory)
      return fail(MLA_ERR_INVALID_ARG, "mla_linear: row stride %lld must be a multiple of 8 elements, at least %lld",
                  static_cast<long long>(strides[i]), static_cast<long long>(widths[i]));
  if (!aligned_to(x, 16) || !aligned_to(weight, 16) || !aligned_to(bias, 16) || !aligned_to(residual, 16) || !aligned_to(out, 16) ||
      !aligned_to(status, 4))
    return fail(MLA_ERR_INVALID_ARG, "mla_linear: pointers must be 16-byte aligned");
  const ByteRange y = bytes_at(out, 2 * ((rows - 1) * out_stride + outer));
  const bool in_place = residual == out && residual_stride == out_stride;
  if (overlap(y, bytes_at(x, 2 * ((rows - 1) * x_stride + inner))) ||
      overlap(y, bytes_at(weight, 2ll * inner * outer)) || overlap(y, bytes_at(bias, bias ? 2ll * outer : 0)) ||
      (!in_place && overlap(y, bytes_at(residual, residual ? 2 * ((rows - 1) * residual_stride + outer) : 0))))
    return fail(MLA_ERR_INVALID_ARG, "mla_linear: out overlaps an input other than residual element for element");

  mla::GemmParams g;
  std::memset(&g, 0, sizeof g);
  g.bias = static_cast<const uint16_t*>(bias);
  g.residual = static_cast<const uint16_t*>(residual);
  g.residual_stride = residual_stride;
  g.out = static_cast<uint16_t*>(out);
  g.out_stride = out_stride;
  g.status = status;
  g.rows = rows;
  g.cols = outer;
  g.k_blocks = (inner + 63) / 64;
  g.act = activation;
  int num_sms = 0;
  if (int rc = mla::current_sm_count(&num_sms)) return rc;
  CUtensorMap x_map, w_map, y_map;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  // Few rows go to the kernel that splits K (64 x 4096 x 4096 in 11.2 us against 16.4 on pairs, 64 x 16384 x 8192 in 46
  // against 62), unless K is too short to be worth its exchange of sums (128 x 512 x 2048: 7.0 against 5.5, 64 x 1544 x 6152:
  // 10.3 against 9.8).
  if (rows <= 32 || (rows <= 128 && g.k_blocks > 32)) {
    const int nt = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    if (int rc = rows_map("mla_linear: x", &x_map, x, inner, rows, x_stride, 64, nt)) return rc;
    if (int rc = rows_map("mla_linear: weight", &w_map, weight, inner, outer, inner, 64, 128)) return rc;
    const int n_tiles = (outer + 127) / 128;
    g.split = 1;
    // CTAs enough for the SMs (two fit one), with four steps of K each at least: 1 x 16384 x 8192 in 72, 49, 42 and 46 us at 1,
    // 2, 4 and 8
    while (g.split < 8 && static_cast<int64_t>(n_tiles) * g.split < num_sms && g.k_blocks >= 8 * g.split) g.split *= 2;
    e = mla::launch_gemm_narrow(nt, g, x_map, w_map, n_tiles * g.split, s);
  } else {
    if (int rc = rows_map("mla_linear: x", &x_map, x, inner, rows, x_stride, 64, 128)) return rc;
    if (int rc = rows_map("mla_linear: out", &y_map, out, outer, rows, out_stride, 64, 32)) return rc;
    const int64_t pairs = num_sms / 2;
    g.m_tiles = (rows + 255) / 256;
    g.band = 8;
    // The tile's width with the shortest run: rounds over the pairs times a tile's time. That falls slowly with its columns
    // (the steps in K cost nearly the same: 4096 x 4096 x 4096 in 19.3 us a round at 128 columns, 22.3 at 256), so what
    // a narrower tile can win is a round: 1001 x 1544 x 6152 in two rounds, 30.5 us at 256 columns and 27.3 at 192.
    int64_t best = 0, tiles = 0;
    for (int cols = 256; cols >= 128; cols -= 32) {
      const int64_t n = static_cast<int64_t>(g.m_tiles) * ((outer + cols - 1) / cols);
      const int64_t time = (n + pairs - 1) / pairs * (cols + 400);
      if (best == 0 || time < best) {
        best = time;
        tiles = n;
        g.tile_cols = cols;
      }
    }
    if (tiles >= (1ll << 30)) return fail(MLA_ERR_UNSUPPORTED, "mla_linear: too many tiles");
    g.n_tiles = (outer + g.tile_cols - 1) / g.tile_cols;
    if (int rc = rows_map("mla_linear: weight", &w_map, weight, inner, outer, inner, 64, g.tile_cols / 2)) return rc;
    e = mla::launch_gemm_pair(g, x_map, w_map, y_map, static_cast<int>(tiles < pairs ? tiles : pairs), s);
  }
  if (e != cudaSuccess) return cuda_fail(e, "mla_linear: launch");
  return MLA_OK;
}

}  // extern "C"
