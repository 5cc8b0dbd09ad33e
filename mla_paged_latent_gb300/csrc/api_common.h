// Shared by the translation units of the C ABI: failures, layouts, byte ranges, tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace mla {

int fail(int code, const char* fmt, ...);           // sets mla_last_error and returns code
int cuda_fail(cudaError_t e, const char* what);
int layout_geometry(int layout, int page_size, int64_t* row_bytes, int64_t* page_bytes, int* dqk);
int current_sm_count(int* n);

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct ByteRange {
  uintptr_t lo, hi;
};
inline ByteRange bytes_at(const void* p, int64_t n) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + static_cast<uintptr_t>(n)};
}
inline bool overlap(const ByteRange& a, const ByteRange& b) { return a.lo < b.hi && b.lo < a.hi; }

// A tensor map of bf16 elements with 128-byte swizzle and zeros past the extents; strides in bytes, rank - 1 of them.
int encode_bf16_map(const char* what, CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box);

}  // namespace mla
