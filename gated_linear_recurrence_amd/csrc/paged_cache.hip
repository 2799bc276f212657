// Page plan and key/value write of the paged cache (include/paged_attn.h).
//
// Both move a few bytes per token and compute next to nothing, so the plan is
// bound by latency and the write by HBM.
//
// plan_kernel: one launch, no waits between workgroups. Which pages a
// sequence gets follows from two prefix sums over the sequences (pages given
// back, pages taken), so every workgroup forms those sums for itself, in LDS,
// from the lengths (12 bytes a sequence, from L2), and then serves its own
// sequences, one per wave. A page taken is looked up where it comes from: in
// the free list as it was, or, for the entries this call pushes, in the block
// table columns given back (which nothing here writes). So no workgroup reads
// what another one writes.
#include <hip/hip_runtime.h>

#include "paged_common.h"

namespace rglru {
namespace paged {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kScan = 2048;        // prefix entries kept in LDS; beyond, one entry per group of sequences
constexpr int kSliceTokens = 512;  // tokens of one sequence that a wave maps

struct PlanArgs {
  const int32_t* ctx;
  const int32_t* held;
  const int32_t* cu;
  const int32_t* count;
  int32_t* table;
  int32_t* free_pages;
  int32_t* count_out;
  int32_t* slots;
  int32_t* positions;
  int32_t* kv_lens;
  int32_t* held_out;
  int32_t* unserved;
  int64_t T;
  int32_t n_pages;
  int32_t N;
  int32_t width;
  int32_t lps;    // log2(page_size)
  int32_t group;  // sequences per prefix entry
};

struct Need {
  int32_t start, fresh, ctx, have, need, rel, take;
};

__device__ __forceinline__ Need need_of(const PlanArgs& a, int n) {
  Need r;
  const int64_t cap = int64_t(a.width) << a.lps;
  const int64_t c0 = min(max(int64_t(a.cu[n]), int64_t(0)), a.T);
  const int64_t c1 = min(max(int64_t(a.cu[n + 1]), c0), a.T);
  const int64_t ctx = min(max(int64_t(a.ctx[n]), int64_t(0)), cap);
  const int64_t held = min(max(int64_t(a.held[n]), int64_t(0)), cap);
  const int64_t up = (int64_t(1) << a.lps) - 1;
  const int64_t need = (ctx + (c1 - c0) + up) >> a.lps;
  r.start = int32_t(c0);
  r.fresh = int32_t(c1 - c0);
  r.ctx = int32_t(ctx);
  r.have = int32_t((held + up) >> a.lps);
  r.need = int32_t(min(need, int64_t(a.width) + 1));  // width + 1: the row is too short
  r.rel = max(r.have - r.need, 0);
  r.take = r.need > a.width ? 0 : max(r.need - r.have, 0);
  return r;
}

__device__ __forceinline__ int64_t wave_inclusive(int64_t v, int lane) {
  for (int d = 1; d < 64; d *= 2) {
    const int64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Page number `idx` of the stack after the pages given back were pushed.
__device__ int32_t stack_page(const PlanArgs& a, int64_t idx, int64_t count, const int64_t* rel_before, int entries) {
  if (idx < count) return a.free_pages[idx];
  const int64_t r = idx - count;
  int lo = 0, hi = entries - 1;  // the last entry whose prefix is <= r
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (rel_before[mid] <= r) lo = mid; else hi = mid - 1;
  }
  int64_t left = r - rel_before[lo];
  for (int n = lo * a.group; n < a.N; ++n) {
    const Need d = need_of(a, n);
    if (left < d.rel) return a.table[int64_t(n) * a.width + d.need + left];
    left -= d.rel;
  }
  return 0;  // not reached: idx is below count plus all pages given back
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs a) {
  __shared__ int64_t take_before[kScan], rel_before[kScan];
  __shared__ int64_t part[2][kPlanWaves];
  __shared__ int32_t last_end, missed;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) last_end = 0, missed = 0;

  // Prefix sums of the pages taken and given back, 256 entries at a time.
  const int entries = (a.N + a.group - 1) / a.group;
  int64_t takes = 0, rels = 0;
  for (int e0 = 0; e0 < entries; e0 += kPlanThreads) {
    const int e = e0 + tid;
    int64_t t = 0, r = 0;
    if (e < entries)
      for (int n = e * a.group; n < min((e + 1) * a.group, a.N); ++n) {
        const Need d = need_of(a, n);
        t += d.take;
        r += d.rel;
      }
    const int64_t ti = wave_inclusive(t, lane), ri = wave_inclusive(r, lane);
    if (lane == 63) part[0][wave] = ti, part[1][wave] = ri;
    __syncthreads();
    int64_t tb = takes, rb = rels;
    for (int w = 0; w < kPlanWaves; ++w) {
      if (w < wave) tb += part[0][w], rb += part[1][w];
      takes += part[0][w];
      rels += part[1][w];
    }
    if (e < entries) take_before[e] = tb + ti - t, rel_before[e] = rb + ri - r;
    __syncthreads();
  }
  const int64_t count = min(max(int64_t(a.count[0]), int64_t(0)), int64_t(a.n_pages));
  const int64_t avail = count + rels;

  // The last workgroup counts: what is taken ends where the last served sequence's pages do.
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == 0) {
    int64_t end = 0;
    int miss = 0;
    for (int e = tid; e < entries; e += kPlanThreads) {
      int64_t upto = take_before[e];
      for (int n = e * a.group; n < min((e + 1) * a.group, a.N); ++n) {
        const Need d = need_of(a, n);
        upto += d.take;
        if (d.need > a.width || (d.take > 0 && upto > avail)) ++miss;
        else if (d.take > 0) end = upto;
      }
    }
    for (int d = 32; d > 0; d /= 2) {
      end = max(end, (int64_t)__shfl_xor(end, d));
      miss += __shfl_xor(miss, d);
    }
    if (lane == 0) {
      atomicMax(&last_end, int32_t(min(end, int64_t(INT32_MAX))));
      atomicAdd(&missed, miss);
    }
    __syncthreads();
    if (tid == 0) {
      a.count_out[0] = int32_t(min(max(avail - last_end, int64_t(0)), int64_t(a.n_pages)));
      a.unserved[0] = missed;
    }
  }

  // Padding rows.
  const int64_t threads = int64_t(gridDim.x) * gridDim.y * kPlanThreads;
  const int64_t end = min(max(int64_t(a.cu[a.N]), int64_t(0)), a.T);
  for (int64_t t = end + (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * kPlanThreads + tid; t < a.T; t += threads) {
    a.slots[t] = -1;
    a.positions[t] = -1;
  }

  for (int64_t n = int64_t(blockIdx.x) * kPlanWaves + wave; n < a.N; n += int64_t(gridDim.x) * kPlanWaves) {
    const Need d = need_of(a, int(n));
    const int e = int(n) / a.group;
    int64_t tb = take_before[e], rb = rel_before[e];
    for (int m = e * a.group; m < n; ++m) {
      const Need o = need_of(a, m);
      tb += o.take;
      rb += o.rel;
    }
    const bool served = d.need <= a.width && (d.take == 0 || tb + d.take <= avail);
    int32_t* row = a.table + n * a.width;
    if (blockIdx.y == 0) {
      for (int j = lane; j < d.rel; j += 64)
        if (count + rb + j < a.n_pages) a.free_pages[count + rb + j] = row[d.need + j];
      if (served)
        for (int j = lane; j < d.take; j += 64)
          row[d.have + j] = stack_page(a, avail - 1 - (tb + j), count, rel_before, entries);
      if (lane == 0) {
        a.kv_lens[n] = served ? d.ctx + d.fresh : d.ctx;
        a.held_out[n] = served ? d.ctx + d.fresh : a.held[n];
      }
    }
    for (int64_t i = int64_t(blockIdx.y) * kSliceTokens; i < d.fresh; i += int64_t(gridDim.y) * kSliceTokens) {
      for (int64_t k = i + lane; k < min(i + kSliceTokens, int64_t(d.fresh)); k += 64) {
        const int64_t pos = d.ctx + k;
        int32_t slot = -1;
        if (served) {
          const int32_t col = int32_t(pos >> a.lps);
          const int32_t page =
              col < d.have ? row[col] : stack_page(a, avail - 1 - (tb + col - d.have), count, rel_before, entries);
          slot = (page << a.lps) + int32_t(pos & ((int64_t(1) << a.lps) - 1));
        }
        a.slots[d.start + k] = slot;
        a.positions[d.start + k] = served ? int32_t(pos) : -1;
      }
    }
  }
}

// One 16-byte piece of a token's keys and the same piece of its values per thread.
constexpr int kWriteThreads = 256;

struct WriteArgs {
  const uint4* k;
  const uint4* v;
  uint4* kc;
  uint4* vc;
  const int32_t* slots;
  int64_t rows16;     // 16-byte pieces from one token to the next in k and v
  int64_t pieces;     // T * per_token
  int64_t n_slots;
  int32_t per_token;  // 16-byte pieces of a token: Hkv * per_row
  int32_t per_row;    // of one head's row
  int32_t heads;
  int32_t lps;
};

__global__ __launch_bounds__(kWriteThreads) void write_kernel(WriteArgs a) {
  const int64_t i = int64_t(blockIdx.x) * kWriteThreads + threadIdx.x;
  if (i >= a.pieces) return;
  const int64_t t = i / a.per_token;
  const int c = int(i - t * a.per_token);
  const int h = c / a.per_row, x = c - h * a.per_row;
  const int32_t slot = a.slots[t];
  if (slot < 0 || slot >= a.n_slots) return;
  const int64_t page = slot >> a.lps, off = slot & ((1 << a.lps) - 1);
  const int64_t dst = (((page * a.heads + h) << a.lps) + off) * a.per_row + x;
  const int64_t src = t * a.rows16 + c;
  const uint4 kk = a.k[src], vv = a.v[src];
  a.kc[dst] = kk;
  a.vc[dst] = vv;
}

}  // namespace
}  // namespace paged
}  // namespace rglru

using namespace rglru;

extern "C" rglru_status_t rglru_page_plan(const rglru_paged_shape_t* sp, const int32_t* context_lens,
                                          const int32_t* held_lens, const int32_t* cu_seqlens, int32_t* block_table,
                                          int32_t* free_pages, const int32_t* free_count, int32_t* free_count_out,
                                          int32_t* slot_map, int32_t* positions, int32_t* kv_lens, int32_t* held_lens_out,
                                          int32_t* unserved, void* stream) {
  if (sp == nullptr) return RGLRU_ERR_INVALID_ARGUMENT;
  const rglru_paged_shape_t s = *sp;
  if (!paged::valid_pages(s) || !paged::valid_table(s)) return RGLRU_ERR_INVALID_ARGUMENT;
  if (context_lens == nullptr || cu_seqlens == nullptr || block_table == nullptr || free_pages == nullptr ||
      free_count == nullptr || free_count_out == nullptr || kv_lens == nullptr || held_lens_out == nullptr || unserved == nullptr ||
      (s.n_tokens > 0 && (slot_map == nullptr || positions == nullptr)) || free_count == free_count_out)
    return RGLRU_ERR_INVALID_ARGUMENT;
  const void* all[] = {context_lens, held_lens,      cu_seqlens, block_table, free_pages, free_count,
                       slot_map,     free_count_out, positions,  kv_lens,     held_lens_out, unserved};
  for (const void* p : all)
    if (!aligned_to(p, 4)) return RGLRU_ERR_MISALIGNED;
  const int64_t tokens = s.n_tokens * 4, seqs = int64_t(s.n_seqs) * 4;
  const paged::Bytes outs[] = {{block_table, seqs * s.max_pages}, {free_pages, s.n_pages * 4}, {free_count_out, 4},
                               {slot_map, tokens},                {positions, tokens},         {kv_lens, seqs},
                               {held_lens_out, seqs},             {unserved, 4}};
  const paged::Bytes ins[] = {{context_lens, seqs}, {held_lens, seqs}, {cu_seqlens, seqs + 4}, {free_count, 4}};
  if (paged::outputs_overlap(outs, ins)) return RGLRU_ERR_INVALID_ARGUMENT;
  paged::PlanArgs a;
  a.ctx = context_lens;
  a.held = held_lens != nullptr ? held_lens : context_lens;
  a.cu = cu_seqlens;
  a.count = free_count;
  a.table = block_table;
  a.free_pages = free_pages;
  a.count_out = free_count_out;
  a.slots = slot_map;
  a.positions = positions;
  a.kv_lens = kv_lens;
  a.held_out = held_lens_out;
  a.unserved = unserved;
  a.T = s.n_tokens;
  a.n_pages = int32_t(s.n_pages);
  a.N = s.n_seqs;
  a.width = s.max_pages;
  a.lps = paged::log2_of(s.page_size);
  a.group = int32_t(ceil_div(s.n_seqs, paged::kScan));
  // A wave per sequence, up to 1024 workgroups, and a row of workgroups per slice of the longest sequence.
  const int64_t longest = s.max_new > 0 ? (s.max_new < s.n_tokens ? s.max_new : s.n_tokens) : s.n_tokens;
  int64_t gx = ceil_div(s.n_seqs, paged::kPlanWaves);
  if (gx > 1024) gx = 1024;
  int64_t gy = ceil_div(longest, paged::kSliceTokens);
  const int64_t most = 2048 / gx > 1 ? 2048 / gx : 1;
  if (gy > most) gy = most;
  if (gy < 1) gy = 1;
  paged::plan_kernel<<<dim3(unsigned(gx), unsigned(gy)), paged::kPlanThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
  return launch_status();
}

extern "C" rglru_status_t rglru_paged_kv_write(const rglru_paged_shape_t* sp, const void* k, const void* v,
                                               void* k_cache, void* v_cache, const int32_t* slot_map, void* stream) {
  if (sp == nullptr) return RGLRU_ERR_INVALID_ARGUMENT;
  const rglru_paged_shape_t s = *sp;
  if (!paged::valid_pages(s) || !paged::valid_io(s) || s.kv_heads < 1 || s.kv_heads > (1 << 14) || s.head_dim < 1 ||
      s.head_dim > (1 << 16))
    return RGLRU_ERR_INVALID_ARGUMENT;
  const int64_t esize = s.io_dtype == RGLRU_IO_BF16 ? 2 : 4;
  const int64_t dense = int64_t(s.kv_heads) * s.head_dim;
  const int64_t stride = paged::row_stride(s.kv_stride, dense);
  if (stride < 0) return RGLRU_ERR_INVALID_ARGUMENT;
  if (s.head_dim * esize % 16 != 0) return RGLRU_ERR_UNSUPPORTED;
  const int64_t per_token = dense * esize / 16;
  const int64_t pieces = s.n_tokens * per_token;
  if (ceil_div(pieces, paged::kWriteThreads) * paged::kWriteThreads >= (int64_t(1) << 32)) return RGLRU_ERR_INVALID_ARGUMENT;
  if (s.n_tokens > 0 && (k == nullptr || v == nullptr || k_cache == nullptr || v_cache == nullptr || slot_map == nullptr))
    return RGLRU_ERR_INVALID_ARGUMENT;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(slot_map, 4) || stride * esize % 16 != 0)
    return RGLRU_ERR_MISALIGNED;
  if (pieces == 0) return RGLRU_OK;
  const int64_t cache = s.n_pages * s.page_size * dense * esize, rows = paged::rows_size(s.n_tokens, stride, dense, esize);
  const paged::Bytes outs[] = {{k_cache, cache}, {v_cache, cache}};
  const paged::Bytes ins[] = {{k, rows}, {v, rows}, {slot_map, s.n_tokens * 4}};
  if (paged::outputs_overlap(outs, ins)) return RGLRU_ERR_INVALID_ARGUMENT;
  paged::WriteArgs a;
  a.k = static_cast<const uint4*>(k);
  a.v = static_cast<const uint4*>(v);
  a.kc = static_cast<uint4*>(k_cache);
  a.vc = static_cast<uint4*>(v_cache);
  a.slots = slot_map;
  a.rows16 = stride * esize / 16;
  a.pieces = pieces;
  a.n_slots = s.n_pages * s.page_size;
  a.per_token = int32_t(per_token);
  a.per_row = int32_t(s.head_dim * esize / 16);
  a.heads = s.kv_heads;
  a.lps = paged::log2_of(s.page_size);
  paged::write_kernel<<<unsigned(ceil_div(pieces, paged::kWriteThreads)), paged::kWriteThreads, 0,
                        static_cast<hipStream_t>(stream)>>>(a);
  return launch_status();
}
