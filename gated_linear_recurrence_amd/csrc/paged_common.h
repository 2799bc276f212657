// Argument checks shared by the paged-cache entry points.
#pragma once

#include <cmath>

#include "common.h"
#include "paged_attn.h"

namespace rglru {
namespace paged {

constexpr int kMaxSeqs = 1 << 16;

inline int log2_of(int32_t p) { return 31 - __builtin_clz(static_cast<unsigned>(p)); }

inline bool valid_pages(const rglru_paged_shape_t& s) {
  const int64_t lim = int64_t(1) << 31;
  return s.n_tokens >= 0 && s.n_tokens < lim && s.page_size >= 8 && s.page_size <= 1024 &&
         (s.page_size & (s.page_size - 1)) == 0 && s.n_pages >= 1 && s.n_pages < lim / s.page_size;
}

inline bool valid_table(const rglru_paged_shape_t& s) {
  return s.n_seqs >= 1 && s.n_seqs <= kMaxSeqs && s.max_pages >= 1 &&
         s.max_pages <= ((int64_t(1) << 31) - (1 << 16)) / s.page_size && s.max_new >= 0;  // tiles may reach past the end
}

inline bool valid_io(const rglru_paged_shape_t& s) {
  return s.io_dtype == RGLRU_IO_F32 || s.io_dtype == RGLRU_IO_BF16;
}

// The stride of a row of `dense` elements, or -1 for one that is too short or too long to index.
inline int64_t row_stride(int64_t stride, int64_t dense) {
  if (stride == 0) return dense;
  return stride < dense || stride >= (int64_t(1) << 31) ? -1 : stride;
}

}  // namespace paged
}  // namespace rglru
