// Write and read-back of the 4-bit paged cache (include/paged_q4.h).
//
// Both are bound by HBM: a block of 32 elements costs 64 bytes of bf16 and 17
// of the cache. 16 200 tokens of 8 heads of 128, keys and values: in bf16 the write 15.2 to 16.7 us, the read-back 16.1 to 16.5 (4.5
// to 4.9 TB/s), in float32 23.8 and 26.9 (5.9 and 5.3 TB/s). A thread holds 8 elements of a row (16 bytes of bf16), four
// neighbours a block: its largest magnitude takes two DPP steps on the bits
// (as integers, so that infinities and NaN stay the largest), its power a few
// integer operations, its codes one conversion instruction for two elements:
// v_cvt_scalef32_pk_fp4_f32 divides by the power and rounds to the nearest
// code, a half to the even one, and v_cvt_scalef32_pk_bf16_fp4 gives the values
// back, NaN for an exponent of 255 (checked over all codes and powers).
#include <hip/hip_runtime.h>

#include "paged_common.h"
#include "paged_q4.h"

namespace rglru {
namespace paged {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kPiece = 8;  // elements of a thread

struct Q4Args {
  const void* k;    // rows of io; written by the read-back
  const void* v;
  uint8_t* kc;
  uint8_t* ks;
  uint8_t* vc;
  uint8_t* vs;
  const int32_t* slots;
  int64_t row;      // elements from one token of k and v to the next
  int64_t pieces;   // T * per_token
  int64_t n_slots;
  int32_t per_token, per_row;  // pieces of a token and of one head's row
  int32_t heads, lps;
};

template <typename E>
__device__ __forceinline__ void load8(const E* from, float* x) {
  const u32x4* p = reinterpret_cast<const u32x4*>(from);
  if constexpr (sizeof(E) == 2) {
    const u32x4 w = p[0];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[2 * j] = __uint_as_float(w[j] << 16), x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  } else {
    const u32x4 a = p[0], b = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(a[j]), x[4 + j] = __uint_as_float(b[j]);
  }
}

// The larger of a value and that of the lane whose number differs in bit 0 (kCtrl 0xB1) or bit 1 (0x4E).
template <int kCtrl>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  const uint32_t o = uint32_t(__builtin_amdgcn_mov_dpp(int(v), kCtrl, 0xF, 0xF, true));
  return v > o ? v : o;
}

// 8 codes of this thread's elements and the byte of its block.
__device__ __forceinline__ uint32_t encode(const float* x, uint32_t& byte) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kPiece; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  top = quad_max<0x4E>(quad_max<0xB1>(top));
  // top = m 2^k with 1 <= m < 2: at most 6 2^e from e = k - 2 on, k - 1 for m past 1.5
  const int e = int(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x400000u);
  const bool odd = top >= 0x7F800000u;
  byte = odd ? 255u : uint32_t(min(max(e, 1), 252));
  const float power = __uint_as_float(byte << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], power, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], power, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], power, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], power, 3);
  return odd ? 0u : w;
}

struct Place {
  int64_t t, row;   // token; row of the cache, [n_pages, Hkv, page_size]
  int32_t h, x;     // head, piece of its row
  bool live;
};
__device__ __forceinline__ Place place_of(const Q4Args& a, int64_t i) {
  Place p;
  p.t = i / a.per_token;
  const int c = int(i - p.t * a.per_token);
  p.h = c / a.per_row;
  p.x = c - p.h * a.per_row;
  const int32_t slot = a.slots[p.t];
  p.live = slot >= 0 && slot < a.n_slots;
  p.row = (((int64_t(p.live ? slot : 0) >> a.lps) * a.heads + p.h) << a.lps) + (slot & ((1 << a.lps) - 1));
  return p;
}

template <typename E>
__global__ __launch_bounds__(kThreads) void write_q4_kernel(Q4Args a) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= a.pieces) return;   // whole blocks: pieces is a multiple of 4
  const Place p = place_of(a, i);
  if (!p.live) return;
  const int64_t src = p.t * a.row + int64_t(p.h * a.per_row + p.x) * kPiece;
  float k[kPiece], v[kPiece];
  load8(static_cast<const E*>(a.k) + src, k);
  load8(static_cast<const E*>(a.v) + src, v);
  uint32_t kb, vb;
  const uint32_t kw = encode(k, kb), vw = encode(v, vb);
  const int64_t at = p.row * a.per_row + p.x;
  reinterpret_cast<uint32_t*>(a.kc)[at] = kw;
  reinterpret_cast<uint32_t*>(a.vc)[at] = vw;
  if (p.x % 4 == 0) {
    a.ks[at / 4] = uint8_t(kb);
    a.vs[at / 4] = uint8_t(vb);
  }
}

// Bits 16 j .. of the result: values 2i + j of the word's byte i, as bf16.
template <int kByte>
__device__ __forceinline__ uint32_t values_of(uint32_t w, float power) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, kByte));
}

template <typename E>
__device__ __forceinline__ void store8(E* to, uint32_t w, uint32_t byte) {
  const float power = __uint_as_float(byte << 23);
  const u32x4 b = {values_of<0>(w, power), values_of<1>(w, power), values_of<2>(w, power), values_of<3>(w, power)};
  u32x4* p = reinterpret_cast<u32x4*>(to);
  if constexpr (sizeof(E) == 2) {
    p[0] = b;
  } else {
    const u32x4 lo = {b[0] << 16, b[0] & 0xFFFF0000u, b[1] << 16, b[1] & 0xFFFF0000u};
    const u32x4 hi = {b[2] << 16, b[2] & 0xFFFF0000u, b[3] << 16, b[3] & 0xFFFF0000u};
    p[0] = lo;
    p[1] = hi;
  }
}

template <typename E>
__global__ __launch_bounds__(kThreads) void read_q4_kernel(Q4Args a, E* k, E* v) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= a.pieces) return;
  const Place p = place_of(a, i);
  const int64_t at = p.row * a.per_row + p.x;
  uint32_t kw = 0, vw = 0, kb = 1, vb = 1;
  if (p.live) {
    kw = reinterpret_cast<const uint32_t*>(a.kc)[at];
    vw = reinterpret_cast<const uint32_t*>(a.vc)[at];
    kb = a.ks[at / 4];
    vb = a.vs[at / 4];
  }
  store8(k + i * kPiece, kw, kb);
  store8(v + i * kPiece, vw, vb);
}

// What both check; `pieces` is the work of the call.
rglru_status_t check(const rglru_paged_shape_t& s, const void* k, const void* v, int64_t stride, const void* kc, const void* ks,
                     const void* vc, const void* vs, const int32_t* slots, int64_t& pieces) {
  if (!valid_pages(s) || !valid_io(s) || s.kv_heads < 1 || s.kv_heads > (1 << 14) || s.head_dim < 1 ||
      s.head_dim > (1 << 16) || stride < 0)
    return RGLRU_ERR_INVALID_ARGUMENT;
  if (s.head_dim % 32 != 0) return RGLRU_ERR_UNSUPPORTED;
  const int64_t esize = s.io_dtype == RGLRU_IO_BF16 ? 2 : 4, dense = int64_t(s.kv_heads) * s.head_dim;
  pieces = s.n_tokens * dense / kPiece;
  if (s.n_tokens * dense * esize > (int64_t(1) << 36) - (1 << 12)) return RGLRU_ERR_INVALID_ARGUMENT;
  if (s.n_tokens > 0 && (k == nullptr || v == nullptr || kc == nullptr || ks == nullptr || vc == nullptr || vs == nullptr ||
                         slots == nullptr))
    return RGLRU_ERR_INVALID_ARGUMENT;
  const void* all[] = {k, v, kc, ks, vc, vs};
  for (const void* p : all)
    if (!aligned_to(p, 16)) return RGLRU_ERR_MISALIGNED;
  if (!aligned_to(slots, 4) || stride * esize % 16 != 0) return RGLRU_ERR_MISALIGNED;
  return RGLRU_OK;
}

Q4Args args_of(const rglru_paged_shape_t& s, const void* k, const void* v, int64_t stride, uint8_t* kc, uint8_t* ks,
               uint8_t* vc, uint8_t* vs, const int32_t* slots, int64_t pieces) {
  Q4Args a;
  a.k = k;
  a.v = v;
  a.kc = kc;
  a.ks = ks;
  a.vc = vc;
  a.vs = vs;
  a.slots = slots;
  a.row = stride;
  a.pieces = pieces;
  a.n_slots = s.n_pages * s.page_size;
  a.per_row = s.head_dim / kPiece;
  a.per_token = s.kv_heads * a.per_row;
  a.heads = s.kv_heads;
  a.lps = log2_of(s.page_size);
  return a;
}

}  // namespace
}  // namespace paged
}  // namespace rglru

using namespace rglru;

extern "C" rglru_status_t rglru_paged_kv_write_q4(const rglru_paged_shape_t* sp, const void* k, const void* v,
                                                  uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes,
                                                  uint8_t* v_scales, const int32_t* slot_map, void* stream) {
  if (sp == nullptr) return RGLRU_ERR_INVALID_ARGUMENT;
  const rglru_paged_shape_t s = *sp;
  const int64_t dense = int64_t(s.kv_heads) * s.head_dim, stride = paged::row_stride(s.kv_stride, dense);
  int64_t pieces;
  const rglru_status_t st = paged::check(s, k, v, stride, k_codes, k_scales, v_codes, v_scales, slot_map, pieces);
  if (st != RGLRU_OK || pieces == 0) return st;
  const int64_t esize = s.io_dtype == RGLRU_IO_BF16 ? 2 : 4, elems = s.n_pages * s.page_size * dense;
  const int64_t rows = paged::rows_size(s.n_tokens, stride, dense, esize);
  const paged::Bytes outs[] = {{k_codes, elems / 2}, {k_scales, elems / 32}, {v_codes, elems / 2}, {v_scales, elems / 32}};
  const paged::Bytes ins[] = {{k, rows}, {v, rows}, {slot_map, s.n_tokens * 4}};
  if (paged::outputs_overlap(outs, ins)) return RGLRU_ERR_INVALID_ARGUMENT;
  const paged::Q4Args a = paged::args_of(s, k, v, stride, k_codes, k_scales, v_codes, v_scales, slot_map, pieces);
  const unsigned grid = unsigned(ceil_div(pieces, paged::kThreads));
  if (s.io_dtype == RGLRU_IO_BF16)
    paged::write_q4_kernel<uint16_t><<<grid, paged::kThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
  else
    paged::write_q4_kernel<float><<<grid, paged::kThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
  return launch_status();
}

extern "C" rglru_status_t rglru_paged_kv_read_q4(const rglru_paged_shape_t* sp, const uint8_t* k_codes,
                                                 const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
                                                 const int32_t* slot_map, void* k, void* v, void* stream) {
  if (sp == nullptr) return RGLRU_ERR_INVALID_ARGUMENT;
  const rglru_paged_shape_t s = *sp;
  const int64_t dense = int64_t(s.kv_heads) * s.head_dim;
  int64_t pieces;
  const rglru_status_t st = paged::check(s, k, v, dense, k_codes, k_scales, v_codes, v_scales, slot_map, pieces);
  if (st != RGLRU_OK || pieces == 0) return st;
  const int64_t esize = s.io_dtype == RGLRU_IO_BF16 ? 2 : 4, elems = s.n_pages * s.page_size * dense;
  const paged::Bytes outs[] = {{k, s.n_tokens * dense * esize}, {v, s.n_tokens * dense * esize}};
  const paged::Bytes ins[] = {{k_codes, elems / 2}, {k_scales, elems / 32}, {v_codes, elems / 2}, {v_scales, elems / 32},
                              {slot_map, s.n_tokens * 4}};
  if (paged::outputs_overlap(outs, ins)) return RGLRU_ERR_INVALID_ARGUMENT;
  const paged::Q4Args a = paged::args_of(s, nullptr, nullptr, dense, const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(k_scales),
                                         const_cast<uint8_t*>(v_codes), const_cast<uint8_t*>(v_scales), slot_map, pieces);
  const unsigned grid = unsigned(ceil_div(pieces, paged::kThreads));
  if (s.io_dtype == RGLRU_IO_BF16)
    paged::read_q4_kernel<<<grid, paged::kThreads, 0, static_cast<hipStream_t>(stream)>>>(a, static_cast<uint16_t*>(k),
                                                                                          static_cast<uint16_t*>(v));
  else
    paged::read_q4_kernel<<<grid, paged::kThreads, 0, static_cast<hipStream_t>(stream)>>>(a, static_cast<float*>(k),
                                                                                          static_cast<float*>(v));
  return launch_status();
}
