// Argument checks shared by the paged-cache entry points.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

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

// Bytes that a call reads or writes from `at` on; of strided rows, from the first one's start to the last one's end.
struct Bytes {
  const void* at;
  int64_t size;
};

inline int64_t rows_size(int64_t rows, int64_t stride, int64_t dense, int64_t esize) {
  if (rows == 0) return 0;
  const int64_t elems = (rows - 1) * stride + dense, most = int64_t(1) << 60;  // rows and strides below 2^31: may pass 2^63 bytes
  return (elems < most ? elems : most) * esize;
}

// Whether one of the outputs overlaps another one or an input.
template <size_t kOuts, size_t kIns>
bool outputs_overlap(const Bytes (&outs)[kOuts], const Bytes (&ins)[kIns]) {
  auto meet = [](const Bytes& a, const Bytes& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return a.at != nullptr && b.at != nullptr && a.size > 0 && b.size > 0 &&
           (x <= y ? y - x < uintptr_t(a.size) : x - y < uintptr_t(b.size));
  };
  for (size_t i = 0; i < kOuts; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return true;
    for (const Bytes& in : ins)
      if (meet(outs[i], in)) return true;
  }
  return false;
}

}  // namespace paged
}  // namespace rglru
