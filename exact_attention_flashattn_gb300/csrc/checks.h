// Argument checks and the end of a call, shared by the C-ABI files.
#pragma once

#include <stdint.h>

#include "../../include/bwattn.h"
#include "kernels.h"

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool good(const void* p, uintptr_t n) { return p != nullptr && aligned(p, n); }
inline bool good_or_null(const void* p, uintptr_t n) { return p == nullptr || aligned(p, n); }
inline bool head_dim(int d) { return d == 64 || d == 128 || d == 256; }
// distance between consecutive rows of `width` elements: 16-byte steps, no overlap, a tensor map's limit
inline bool row_stride(int64_t stride, int64_t width) {
  return stride >= width && stride % 8 == 0 && stride < (static_cast<int64_t>(1) << 38);
}
inline bool page_sizes(int page_size, int num_pages) {
  return page_size >= 16 && page_size <= 1024 && page_size % 16 == 0 && num_pages > 0 &&
         static_cast<int64_t>(num_pages) * page_size <= 0x7fffffff;
}
inline int done(cudaError_t e) {
  if (e != cudaSuccess) {
    bw::record_cuda_error(e);
    return BWATTN_ERR_CUDA;
  }
  return BWATTN_OK;
}

}  // namespace
