// Attention of new tokens over a paged key/value cache (include/paged_attn.h).
//
// One wave per row (token, query head): 64 keys at a time, a key per lane for
// the scores, a column of the values per lane for the output, with the running
// maximum and sum of the softmax.
#include <hip/hip_runtime.h>

#include "paged_common.h"

namespace rglru {
namespace paged {

namespace {

struct AttnArgs {
  const int32_t* cu;
  const int32_t* kv_lens;
  const int32_t* table;
  const void* q;
  const void* kc;
  const void* vc;
  void* o;
  float* lse;
  int64_t T, q_stride;
  int32_t n_pages, N, width, lps, Hq, Hkv, window;
  float scale;
};

__device__ __forceinline__ float load1(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load1(const uint16_t* p, int64_t i) { return bf16_bits_to_f32(p[i]); }
__device__ __forceinline__ void store1(float* p, int64_t i, float f) { p[i] = f; }
__device__ __forceinline__ void store1(uint16_t* p, int64_t i, float f) { p[i] = f32_to_bf16(f); }

template <typename E, int D>
__global__ __launch_bounds__(256) void attn_kernel(AttnArgs a) {
  __shared__ float qs[4][D], ps[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r = int64_t(blockIdx.x) * 4 + wave;
  const int64_t t = r / a.Hq;
  if (t >= min(max(int64_t(a.cu[a.N]), int64_t(0)), a.T)) return;
  const int h = int(r - t * a.Hq), hk = h / (a.Hq / a.Hkv);
  int lo = 0, hi = a.N - 1;  // the last sequence that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int64_t kv = min(max(int64_t(a.kv_lens[lo]), int64_t(0)), int64_t(a.width) << a.lps);
  const int64_t pos = kv - (int64_t(a.cu[lo + 1]) - t);
  const int64_t first = a.window > 0 ? max(pos - a.window + 1, int64_t(0)) : 0;
  const E* q = static_cast<const E*>(a.q) + t * a.q_stride + int64_t(h) * D;
  for (int d = lane; d < D; d += 64) qs[wave][d] = load1(q, d);
  float acc[D / 64] = {}, m = -INFINITY, l = 0.0f;
  for (int64_t j0 = first; j0 <= min(pos, kv - 1); j0 += 64) {
    const int64_t j = j0 + lane;
    const bool seen = j <= pos && j < kv;
    float s = -INFINITY;
    if (seen) {
      const int64_t page = min(max(a.table[int64_t(lo) * a.width + (j >> a.lps)], 0), a.n_pages - 1);
      const E* k = static_cast<const E*>(a.kc) + ((((page * a.Hkv + hk) << a.lps) + (j & ((1 << a.lps) - 1))) * D);
      float dot = 0.0f;
      for (int d = 0; d < D; ++d) dot += qs[wave][d] * load1(k, d);
      s = dot * a.scale;
    }
    float top = s;
    for (int x = 32; x > 0; x /= 2) top = fmaxf(top, __shfl_xor(top, x));
    const float m_new = fmaxf(m, top), base = m_new == -INFINITY ? 0.0f : m_new;
    const float p = seen ? __expf(s - base) : 0.0f, keep = __expf(m - base);
    float sum = p;
    for (int x = 32; x > 0; x /= 2) sum += __shfl_xor(sum, x);
    l = l * keep + sum;
    m = m_new;
    ps[wave][lane] = p;
    for (int c = 0; c < D / 64; ++c) acc[c] *= keep;
    const int n = int(min(int64_t(64), min(pos, kv - 1) - j0 + 1));
    for (int x = 0; x < n; ++x) {
      const int64_t jj = j0 + x;
      const int64_t page = min(max(a.table[int64_t(lo) * a.width + (jj >> a.lps)], 0), a.n_pages - 1);
      const E* v = static_cast<const E*>(a.vc) + ((((page * a.Hkv + hk) << a.lps) + (jj & ((1 << a.lps) - 1))) * D);
      for (int c = 0; c < D / 64; ++c) acc[c] += ps[wave][x] * load1(v, c * 64 + lane);
    }
  }
  E* o = static_cast<E*>(a.o) + r * D;
  const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
  for (int c = 0; c < D / 64; ++c) store1(o, c * 64 + lane, m == -INFINITY ? 0.0f : acc[c] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[r] = m == -INFINITY ? -INFINITY : m + logf(l);
}

rglru_status_t check(const rglru_paged_shape_t& s) {
  if (!valid_pages(s) || !valid_table(s) || !valid_io(s) || s.kv_heads < 1 || s.q_heads < s.kv_heads ||
      s.q_heads > (1 << 14) || s.q_heads % s.kv_heads != 0 || s.n_tokens * s.q_heads >= (int64_t(1) << 31) ||
      s.head_dim < 1 || s.head_dim > (1 << 16) || s.window < 0 || !std::isfinite(s.scale) ||
      row_stride(s.q_stride, int64_t(s.q_heads) * s.head_dim) < 0)
    return RGLRU_ERR_INVALID_ARGUMENT;
  if (s.head_dim != 64 && s.head_dim != 128 && s.head_dim != 256) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

template <typename E>
void launch(const AttnArgs& a, int dim, hipStream_t st) {
  const unsigned grid = unsigned(ceil_div(a.T * a.Hq, 4));
  if (dim == 64) attn_kernel<E, 64><<<grid, 256, 0, st>>>(a);
  else if (dim == 128) attn_kernel<E, 128><<<grid, 256, 0, st>>>(a);
  else attn_kernel<E, 256><<<grid, 256, 0, st>>>(a);
}

}  // namespace
}  // namespace paged
}  // namespace rglru

using namespace rglru;

extern "C" size_t rglru_paged_attn_workspace_bytes(const rglru_paged_shape_t* sp) {
  if (sp == nullptr || paged::check(*sp) != RGLRU_OK) return 0;
  return 256;
}

extern "C" rglru_status_t rglru_paged_attn_fwd(const rglru_paged_shape_t* sp, const int32_t* cu_seqlens,
                                               const int32_t* kv_lens, const int32_t* block_table, const void* q,
                                               const void* k_cache, const void* v_cache, void* o, float* lse,
                                               void* workspace, size_t workspace_bytes, void* stream) {
  if (sp == nullptr) return RGLRU_ERR_INVALID_ARGUMENT;
  const rglru_paged_shape_t s = *sp;
  const rglru_status_t st = paged::check(s);
  if (st == RGLRU_ERR_INVALID_ARGUMENT) return st;
  if (s.n_tokens > 0 && (cu_seqlens == nullptr || kv_lens == nullptr || block_table == nullptr || q == nullptr ||
                         k_cache == nullptr || v_cache == nullptr || o == nullptr || workspace == nullptr))
    return RGLRU_ERR_INVALID_ARGUMENT;
  if (st != RGLRU_OK) return st;
  const int64_t stride = paged::row_stride(s.q_stride, int64_t(s.q_heads) * s.head_dim);
  const int64_t esize = s.io_dtype == RGLRU_IO_BF16 ? 2 : 4;
  if (!aligned_to(cu_seqlens, 4) || !aligned_to(kv_lens, 4) || !aligned_to(block_table, 4) || !aligned_to(q, 16) ||
      !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(o, 16) || !aligned_to(lse, 4) ||
      !aligned_to(workspace, 256) || stride * esize % 16 != 0)
    return RGLRU_ERR_MISALIGNED;
  if (s.n_tokens == 0) return RGLRU_OK;
  if (workspace_bytes < rglru_paged_attn_workspace_bytes(&s)) return RGLRU_ERR_WORKSPACE_TOO_SMALL;
  paged::AttnArgs a;
  a.cu = cu_seqlens;
  a.kv_lens = kv_lens;
  a.table = block_table;
  a.q = q;
  a.kc = k_cache;
  a.vc = v_cache;
  a.o = o;
  a.lse = lse;
  a.T = s.n_tokens;
  a.q_stride = stride;
  a.n_pages = int32_t(s.n_pages);
  a.N = s.n_seqs;
  a.width = s.max_pages;
  a.lps = paged::log2_of(s.page_size);
  a.Hq = s.q_heads;
  a.Hkv = s.kv_heads;
  a.window = s.window;
  a.scale = s.scale;
  if (s.io_dtype == RGLRU_IO_BF16) paged::launch<uint16_t>(a, s.head_dim, static_cast<hipStream_t>(stream));
  else paged::launch<float>(a, s.head_dim, static_cast<hipStream_t>(stream));
  return launch_status();
}
