// Attention of new tokens over a 4-bit paged cache (include/paged_q4.h).
//
// The simplest kernel: a wave per row (token, query head), 64 keys at a time, a
// key per lane for the scores, D / 64 columns per lane for the values, with the
// running maximum and sum of the softmax in float32.
#include <hip/hip_runtime.h>

#include "paged_common.h"
#include "paged_q4.h"

namespace rglru {
namespace paged {

namespace {

struct Attn4Args {
  const int32_t* cu;
  const int32_t* kv_lens;
  const int32_t* table;
  const void* q;
  const uint8_t* kc;
  const uint8_t* ks;
  const uint8_t* vc;
  const uint8_t* vs;
  void* o;
  float* lse;
  int64_t q_stride;
  int32_t T, n_pages, N, width, lps, Hq, Hkv, group, window;
  float scale;
};

__device__ __forceinline__ float value_of(uint32_t code, uint32_t byte) {
  const float half[8] = {0.0f, 0.5f, 1.0f, 1.5f, 2.0f, 3.0f, 4.0f, 6.0f};
  if (byte == 255u) return __uint_as_float(0x7FC00000u);
  const float x = ldexpf(half[code & 7], int(byte) - 127);
  return code & 8 ? -x : x;
}

template <typename E>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (sizeof(E) == 2) return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

template <typename E, int D>
__global__ __launch_bounds__(64) void attn_q4_simple(Attn4Args a) {
  __shared__ float qs[D];
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int32_t t = int32_t(row / a.Hq), hq = int32_t(row - int64_t(t) * a.Hq), hk = hq / a.group;
  int lo = 0, hi = a.N;   // the first sequence that ends behind t
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.cu[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  if (lo >= a.N) return;
  const int32_t start = min(max(a.cu[lo], 0), a.T), end = min(max(a.cu[lo + 1], start), a.T);
  if (t < start || t >= end) return;
  const int32_t kv = min(max(a.kv_lens[lo], 0), a.width << a.lps);
  const int32_t last = max(kv - (end - start) + (t - start), -1), first = a.window > 0 ? max(last - a.window + 1, 0) : 0;
  for (int d = lane; d < D; d += 64) qs[d] = load1<E>(a.q, t * a.q_stride + int64_t(hq) * D + d);
  __syncthreads();
  float m = -INFINITY, l = 0.0f, o[D / 64] = {};
  const int32_t* table = a.table + int64_t(lo) * a.width;
  for (int32_t j0 = first; j0 <= last; j0 += 64) {
    const int32_t j = j0 + lane;
    const int64_t page = min(max(table[min(j, last) >> a.lps], 0), a.n_pages - 1);
    const int64_t at = (((page * a.Hkv + hk) << a.lps) + (min(j, last) & ((1 << a.lps) - 1)));
    float s = -INFINITY;
    if (j <= last) {
      s = 0.0f;
      for (int d = 0; d < D; d += 2) {
        const uint32_t c = a.kc[at * (D / 2) + d / 2], b = a.ks[at * (D / 32) + d / 32];
        s += qs[d] * value_of(c & 15, b) + qs[d + 1] * value_of(c >> 4, b);
      }
      s *= a.scale;
    }
    float top = s;
    bool nan = s != s;
    for (int d = 32; d > 0; d /= 2) top = fmaxf(top, __shfl_xor(top, d)), nan |= bool(__shfl_xor(int(nan), d));
    const float m_new = fmaxf(m, top), base = m_new == -INFINITY ? 0.0f : m_new;
    const float keep = expf(m - base), p = nan ? __uint_as_float(0x7FC00000u) : expf(s - base);
    float sum = p;
    for (int d = 32; d > 0; d /= 2) sum += __shfl_xor(sum, d);
    l = l * keep + sum;
    for (int x = 0; x < D / 64; ++x) o[x] *= keep;
    m = nan && m_new == -INFINITY ? 0.0f : m_new;
    for (int k = 0; k < min(64, last - j0 + 1); ++k) {
      const float w = __shfl(p, k);
      const int64_t v = __shfl(at, k);
      for (int x = 0; x < D / 64; ++x) {
        const int d = x * 64 + lane;
        const uint32_t c = a.vc[v * (D / 2) + d / 2], b = a.vs[v * (D / 32) + d / 32];
        o[x] += w * value_of(d & 1 ? c >> 4 : c & 15, b);
      }
    }
  }
  const bool none = m == -INFINITY;
  for (int x = 0; x < D / 64; ++x) {
    const float r = none ? 0.0f : o[x] / l;
    if constexpr (sizeof(E) == 2) static_cast<uint16_t*>(a.o)[row * D + x * 64 + lane] = f32_to_bf16(r);
    else static_cast<float*>(a.o)[row * D + x * 64 + lane] = r;
  }
  if (a.lse != nullptr && lane == 0) a.lse[row] = none ? -INFINITY : m + logf(l);
}

rglru_status_t check(const rglru_paged_shape_t& s) {
  if (!valid_pages(s) || !valid_table(s) || !valid_io(s) || s.kv_heads < 1 || s.q_heads < s.kv_heads ||
      s.q_heads > (1 << 14) || s.q_heads % s.kv_heads != 0 || s.n_tokens * s.q_heads > (int64_t(1) << 31) - (1 << 16) ||
      s.head_dim < 1 || s.head_dim > (1 << 16) || s.window < 0 || !std::isfinite(std::fabs(s.scale) * 1.4426950408889634f) ||
      row_stride(s.q_stride, int64_t(s.q_heads) * s.head_dim) < 0)
    return RGLRU_ERR_INVALID_ARGUMENT;
  if (s.head_dim != 64 && s.head_dim != 128 && s.head_dim != 256) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

}  // namespace
}  // namespace paged
}  // namespace rglru

using namespace rglru;

extern "C" size_t rglru_paged_attn_q4_workspace_bytes(const rglru_paged_shape_t* sp) {
  return sp == nullptr || paged::check(*sp) != RGLRU_OK ? 0 : 256;
}

extern "C" rglru_status_t rglru_paged_attn_q4_fwd(const rglru_paged_shape_t* sp, const int32_t* cu_seqlens,
                                                  const int32_t* kv_lens, const int32_t* block_table, const void* q,
                                                  const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                                                  const uint8_t* v_scales, void* o, float* lse, void* workspace,
                                                  size_t workspace_bytes, void* stream) {
  if (sp == nullptr) return RGLRU_ERR_INVALID_ARGUMENT;
  const rglru_paged_shape_t s = *sp;
  const rglru_status_t st = paged::check(s);
  if (st == RGLRU_ERR_INVALID_ARGUMENT) return st;
  if (s.n_tokens > 0 && (cu_seqlens == nullptr || kv_lens == nullptr || block_table == nullptr || q == nullptr ||
                         k_codes == nullptr || k_scales == nullptr || v_codes == nullptr || v_scales == nullptr ||
                         o == nullptr || workspace == nullptr))
    return RGLRU_ERR_INVALID_ARGUMENT;
  if (st != RGLRU_OK) return st;
  const int64_t stride = paged::row_stride(s.q_stride, int64_t(s.q_heads) * s.head_dim);
  const int64_t esize = s.io_dtype == RGLRU_IO_BF16 ? 2 : 4;
  if (!aligned_to(cu_seqlens, 4) || !aligned_to(kv_lens, 4) || !aligned_to(block_table, 4) || !aligned_to(q, 16) ||
      !aligned_to(k_codes, 16) || !aligned_to(k_scales, 16) || !aligned_to(v_codes, 16) || !aligned_to(v_scales, 16) ||
      !aligned_to(o, 16) || !aligned_to(lse, 4) || !aligned_to(workspace, 256) || stride * esize % 16 != 0)
    return RGLRU_ERR_MISALIGNED;
  if (s.n_tokens == 0) return RGLRU_OK;
  const size_t need = rglru_paged_attn_q4_workspace_bytes(&s);
  if (workspace_bytes < need) return RGLRU_ERR_WORKSPACE_TOO_SMALL;
  const int64_t dense = int64_t(s.q_heads) * s.head_dim, seqs = int64_t(s.n_seqs) * 4;
  const int64_t cache = s.n_pages * s.page_size * s.kv_heads * s.head_dim;
  const paged::Bytes outs[] = {{o, s.n_tokens * dense * esize}, {lse, s.n_tokens * s.q_heads * 4}, {workspace, int64_t(need)}};
  const paged::Bytes ins[] = {{cu_seqlens, seqs + 4}, {kv_lens, seqs},        {block_table, seqs * s.max_pages},
                              {q, paged::rows_size(s.n_tokens, stride, dense, esize)}, {k_codes, cache / 2},
                              {k_scales, cache / 32}, {v_codes, cache / 2},   {v_scales, cache / 32}};
  if (paged::outputs_overlap(outs, ins)) return RGLRU_ERR_INVALID_ARGUMENT;
  paged::Attn4Args a = {cu_seqlens, kv_lens, block_table, q, k_codes, k_scales, v_codes, v_scales, o, lse, stride,
                        int32_t(s.n_tokens), int32_t(s.n_pages), s.n_seqs, s.max_pages, paged::log2_of(s.page_size), s.q_heads,
                        s.kv_heads, s.q_heads / s.kv_heads, s.window, s.scale};
  const unsigned grid = unsigned(s.n_tokens * s.q_heads);
  const hipStream_t h = static_cast<hipStream_t>(stream);
  const bool b = s.io_dtype == RGLRU_IO_BF16;
  if (s.head_dim == 64) b ? paged::attn_q4_simple<uint16_t, 64><<<grid, 64, 0, h>>>(a) : paged::attn_q4_simple<float, 64><<<grid, 64, 0, h>>>(a);
  else if (s.head_dim == 128) b ? paged::attn_q4_simple<uint16_t, 128><<<grid, 64, 0, h>>>(a) : paged::attn_q4_simple<float, 128><<<grid, 64, 0, h>>>(a);
  else b ? paged::attn_q4_simple<uint16_t, 256><<<grid, 64, 0, h>>>(a) : paged::attn_q4_simple<float, 256><<<grid, 64, 0, h>>>(a);
  return launch_status();
}
