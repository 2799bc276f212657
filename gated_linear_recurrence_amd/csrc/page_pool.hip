// Fork, free, compact and copy of a pool of cache pages (include/page_pool.h).
//
// The first three move a few bytes for every page that they touch, so they are
// bound by latency: what counts is the number of launches and, in each, of
// dependent reads. Whole numbers only, so the results do not depend on timing:
// counts of sharing change by atomics, whose order does not matter, and every
// place in a list comes from a prefix sum in the order of rows or pages. No
// workgroup waits for another one; what needs the sums of all goes into the
// next launch.
#include <hip/hip_runtime.h>

#include "page_pool.h"
#include "paged_common.h"

namespace rglru {
namespace paged {

namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = kThreads / 64;

// Sum over the lanes before this one, itself included.
__device__ __forceinline__ int32_t wave_inclusive(int32_t v, int lane) {
  for (int d = 1; d < 64; d *= 2) {
    const int32_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The same over the threads of a workgroup; `total` is the sum of all. `part`: a word of LDS for every wave.
template <int kAll = kThreads>
__device__ __forceinline__ int32_t block_inclusive(int32_t v, int32_t* part, int32_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  v = wave_inclusive(v, lane);
  __syncthreads();
  if (lane == 63) part[wave] = v;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kAll / 64; ++w) {
    if (w < wave) v += part[w];
    total += part[w];
  }
  return v;
}

__device__ __forceinline__ int32_t block_sum(int32_t v, int32_t* part) {
  int32_t total;
  block_inclusive(v, part, total);
  return total;
}

// The kernels that hold a bit for every page in LDS (see small_free and small_compact).
constexpr int kSmallThreads = 1024;

// The pages of a word from `first` on.
__device__ __forceinline__ uint32_t bits_from(int word, int32_t first) {
  const int32_t p0 = word * 32;
  return first <= p0 ? ~0u : first >= p0 + 32 ? 0u : ~0u << (first - p0);
}

struct Rows {
  const int32_t* table;
  int32_t n_pages, N, width, lps;
};

__device__ __forceinline__ int32_t pages_of(const Rows& r, int32_t tokens) {
  const int64_t t = min(max(int64_t(tokens), int64_t(0)), int64_t(r.width) << r.lps);
  return int32_t((t + (int64_t(1) << r.lps) - 1) >> r.lps);
}

// ---- fork ----
//
// One launch: a page is popped at most once a row, so a row's place in the list
// is the number of rows before it that ask for one, which every workgroup counts
// for itself (16 bytes a row, from L2) before it serves its own rows, one per wave.
// 5.5 us for 64 answers to 8 questions of up to 2000 tokens in pages of 16, 6.2 for 256
// rows of 512.
struct ForkArgs {
  Rows r;
  const int32_t* from;
  const int32_t* lens;
  const int32_t* held;
  const int32_t* free_pages;
  const int32_t* count;
  int32_t* table;
  int32_t* shares;
  int32_t* pairs;
  int32_t* lens_out;
  int32_t* held_out;
  int32_t* count_out;
  int32_t* unserved;
  int32_t rows;  // of a workgroup
};

struct Fork {
  int32_t src, len;
  bool asked, valid, part;  // part: needs a page
};
__device__ __forceinline__ Fork fork_of(const ForkArgs& a, int n) {
  Fork f = {-1, 0, false, false, false};
  const int32_t s = a.from[n];
  if (s < 0) return f;
  f.asked = true;
  f.src = s;
  f.valid = s < a.r.N && s != n && a.lens[n] == 0 && a.held[n] == 0 && a.from[min(s, a.r.N - 1)] < 0;
  if (!f.valid) return f;
  f.len = int32_t(min(max(int64_t(a.lens[s]), int64_t(0)), int64_t(a.r.width) << a.r.lps));
  f.part = (f.len & ((1 << a.r.lps) - 1)) != 0;
  return f;
}

__global__ __launch_bounds__(kThreads) void fork_kernel(ForkArgs a) {
  __shared__ int32_t part[kWaves], ranks[kThreads];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int first = blockIdx.x * a.rows, end = min(first + a.rows, a.r.N);
  const bool last = blockIdx.x == gridDim.x - 1;
  const int32_t count = min(max(a.count[0], 0), a.r.n_pages);
  int32_t mine = 0, bad = 0;
  for (int n = tid; n < (last ? a.r.N : first); n += kThreads) {
    const Fork f = fork_of(a, n);
    mine += f.part && n < first;
    bad += f.asked && !f.valid;
  }
  int32_t before = block_sum(mine, part);
  if (last) bad = block_sum(bad, part);
  for (int n0 = first; n0 < end; n0 += kThreads) {
    const int32_t want = n0 + tid < end ? fork_of(a, n0 + tid).part : 0;
    int32_t total;
    ranks[tid] = before + block_inclusive(want, part, total) - want;
    before += total;
    __syncthreads();
    for (int i = wave; i < min(kThreads, end - n0); i += kWaves) {
      const int n = n0 + i;
      const Fork f = fork_of(a, n);
      const int32_t rank = ranks[i];
      const bool served = f.valid && (!f.part || rank < count);
      int32_t from = -1, to = -1;
      if (served) {
        const int32_t full = f.len >> a.r.lps;
        const int32_t* const src = a.table + int64_t(f.src) * a.r.width;
        int32_t* const dst = a.table + int64_t(n) * a.r.width;
        for (int j = lane; j < full; j += 64) {
          const int32_t p = src[j];
          dst[j] = p;
          if (p >= 0 && p < a.r.n_pages) atomicAdd(a.shares + p, 1);
        }
        if (f.part) {
          from = src[full];
          to = a.free_pages[count - 1 - rank];
          if (lane == 0) dst[full] = to;
        }
      }
      if (lane == 0) {
        a.pairs[2 * int64_t(n)] = from;
        a.pairs[2 * int64_t(n) + 1] = to;
        a.lens_out[n] = served ? f.len : a.lens[n];
        a.held_out[n] = served ? f.len : a.held[n];
      }
    }
    __syncthreads();
  }
  if (last && tid == 0) {
    a.count_out[0] = max(count - before, 0);
    a.unserved[0] = bad + max(before - count, 0);
  }
}

// ---- free ----
//
// Three launches: every row takes its pages' counts down (a page that nobody
// holds any more ends below 0, however often it was given up); chunks of the
// pool count those; and each chunk, which then knows how many lie in the chunks
// after it, writes its own to the list and sets their counts back to 0. 1024 rows of
// up to 8192 tokens in pages of 16, 254 000 pages: 13 us.
constexpr int kEach = 8, kChunk = kThreads * kEach;  // pages of a thread and of a workgroup
constexpr int kSlice = 1024;                         // columns of a row that a wave works on

struct FreeArgs {
  Rows r;
  const int32_t* keep;
  const int32_t* held;
  const int32_t* count;
  int32_t* shares;
  int32_t* free_pages;
  int32_t* held_out;
  int32_t* count_out;
  int32_t* counts;  // of the chunks
  int32_t chunks;
};

__global__ __launch_bounds__(kThreads) void free_mark_kernel(FreeArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t n = int64_t(blockIdx.x) * kWaves + wave; n < a.r.N; n += int64_t(gridDim.x) * kWaves) {
    const int32_t held = a.held[n], kept = min(max(a.keep[n], 0), held);
    const int32_t* const row = a.r.table + n * a.r.width;
    const int32_t stay = pages_of(a.r, kept), have = pages_of(a.r, held);
    for (int64_t j0 = stay + int64_t(blockIdx.y) * kSlice; j0 < have; j0 += int64_t(gridDim.y) * kSlice)
      for (int64_t j = j0 + lane; j < min(j0 + kSlice, int64_t(have)); j += 64) {
        const int32_t p = row[j];
        if (p >= 0 && p < a.r.n_pages) atomicSub(a.shares + p, 1);
      }
    if (blockIdx.y == 0 && lane == 0) a.held_out[n] = kept;
  }
}

// The pages of this thread that nobody holds, as bits.
__device__ __forceinline__ uint32_t gone_of(const FreeArgs& a, int64_t p0) {
  uint32_t gone = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) gone |= uint32_t(p0 + k < a.r.n_pages && a.shares[p0 + k] < 0) << k;
  return gone;
}

__global__ __launch_bounds__(kThreads) void free_count_kernel(FreeArgs a) {
  __shared__ int32_t part[kWaves];
  const int32_t sum = block_sum(__popc(gone_of(a, (int64_t(blockIdx.x) * kThreads + threadIdx.x) * kEach)), part);
  if (threadIdx.x == 0) a.counts[blockIdx.x] = sum;
}

__global__ __launch_bounds__(kThreads) void free_list_kernel(FreeArgs a) {
  __shared__ int32_t part[kWaves];
  const int tid = threadIdx.x;
  int32_t later = 0;
  for (int c = int(blockIdx.x) + 1 + tid; c < a.chunks; c += kThreads) later += a.counts[c];
  const int32_t base = min(max(a.count[0], 0), a.r.n_pages) + block_sum(later, part);
  const int64_t p0 = (int64_t(blockIdx.x) * kThreads + tid) * kEach;
  const uint32_t gone = gone_of(a, p0);
  int32_t total;
  const int32_t upto = block_inclusive(__popc(gone), part, total);
  int32_t at = base + total - upto;   // the pages of later threads come first
#pragma unroll
  for (int k = kEach - 1; k >= 0; --k)
    if (gone >> k & 1) {
      if (at < a.r.n_pages) a.free_pages[at] = int32_t(p0 + k);
      a.shares[p0 + k] = 0;
      ++at;
    }
  if (blockIdx.x == 0 && tid == 0) a.count_out[0] = min(base + total, a.r.n_pages);
}

// Small pools: one workgroup, one launch, a bit in LDS for a page that is freed. The entries that rows give up stand in one
// line, so that every thread has a few to look up beside each other. The first to give a page up marks it, further ones take
// its count down; then every marked page either goes onto the list, its place from the sums over the marks, or has its count
// taken down for the first one. A CU's atomics are slow (8 000 pages given up, 28 000 in the pool: 20 us with two on memory for each, 15 so).
constexpr int kFreePages = 1 << 13, kFreeRows = 64, kFreeEntries = 1 << 14;   // of the pool, of the table
constexpr int kFreeWords = kFreePages / 32;
static_assert(kFreeWords <= kSmallThreads && kFreeRows <= kSmallThreads, "a thread sums up one word, one row");

__global__ __launch_bounds__(kSmallThreads) void free_small_kernel(FreeArgs a) {
  __shared__ uint32_t gone[kFreeWords];
  __shared__ int32_t before[kFreeWords];
  __shared__ int32_t stays[kFreeRows], ends[kFreeRows];   // a row's first entry given up; entries of the rows up to it
  __shared__ int32_t part[kSmallThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, words = (a.r.n_pages + 31) / 32, padded = (a.r.n_pages + 63) / 64 * 64;
  for (int w = tid; w < padded / 32; w += kSmallThreads) gone[w] = 0;
  int32_t given = 0, all;
  if (tid < a.r.N) {
    const int32_t held = a.held[tid], kept = min(max(a.keep[tid], 0), held);
    a.held_out[tid] = kept;
    stays[tid] = pages_of(a.r, kept);
    given = max(pages_of(a.r, held) - stays[tid], 0);
  }
  const int32_t through = block_inclusive<kSmallThreads>(given, part, all);
  if (tid < a.r.N) ends[tid] = through;
  __syncthreads();
  constexpr int kAhead = 4;
  for (int i0 = tid; i0 < all; i0 += kAhead * kSmallThreads) {
    int32_t page[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = min(i0 + k * kSmallThreads, all - 1);
      int lo = 0, hi = a.r.N - 1;   // the first row that ends behind i
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (ends[mid] > i) hi = mid; else lo = mid + 1;
      }
      page[k] = a.r.table[int64_t(lo) * a.r.width + stays[lo] + i - (lo > 0 ? ends[lo - 1] : 0)];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k * kSmallThreads < all && page[k] >= 0 && page[k] < a.r.n_pages) {
        const uint32_t bit = 1u << (page[k] % 32);
        if (atomicOr(gone + page[k] / 32, bit) & bit) atomicSub(a.shares + page[k], 1);
      }
  }
  __threadfence();
  __syncthreads();
  for (int p0 = tid; p0 < padded; p0 += kAhead * kSmallThreads) {
    int32_t shares[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int p = p0 + k * kSmallThreads;
      shares[k] = p < a.r.n_pages && (gone[p / 32] >> (p % 32) & 1) ? a.shares[p] : INT32_MAX;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int p = p0 + k * kSmallThreads;
      if (p >= padded) break;
      const bool marked = p < a.r.n_pages && (gone[p / 32] >> (p % 32) & 1);
      const uint64_t free = __ballot(marked && shares[k] <= 0);
      if (marked && shares[k] != 0) a.shares[p] = max(shares[k] - 1, 0);
      if (lane == 0) gone[p / 32] = uint32_t(free), gone[p / 32 + 1] = uint32_t(free >> 32);
    }
  }
  __syncthreads();
  int32_t total;
  const int32_t mine = tid < words ? __popc(gone[tid]) : 0, upto = block_inclusive<kSmallThreads>(mine, part, total);
  if (tid < words) before[tid] = upto - mine;
  __syncthreads();
  const int32_t count = min(max(a.count[0], 0), a.r.n_pages);
  for (int p = tid; p < a.r.n_pages; p += kSmallThreads) {
    const uint32_t word = gone[p / 32];
    if (!(word >> (p % 32) & 1)) continue;
    const int32_t at = count + total - 1 - (before[p / 32] + __popc(word & ((1u << (p % 32)) - 1)));
    if (at < a.r.n_pages) a.free_pages[at] = p;
  }
  if (tid == 0) a.count_out[0] = min(count + total, a.r.n_pages);
}

// ---- compact ----
//
// Small pools: one launch. Every workgroup marks the pages in use and the free
// ones for itself, in LDS, with the sums before every 32 of them, and writes
// its share of the outputs; where the i-th page moves to is looked up in the sums.
//
// Others, five launches: marks to 0; marks of the pages that rows hold and of those
// on the free list; counts per chunk; ranks, which give the pairs and the new
// list; and the table and the counts of sharing, which follow the ranks.
struct CompactArgs {
  Rows r;
  const int32_t* held;
  const int32_t* shares;
  const int32_t* free_pages;
  const int32_t* count;
  int32_t* table_out;
  int32_t* shares_out;
  int32_t* free_out;
  int32_t* count_out;
  int32_t* pairs;
  int32_t* n_pairs;
  int32_t* unmoved;
  uint8_t* used;    // [n_pages], padded to whole chunks
  uint8_t* idle;    // the same, right behind
  int32_t* counts;  // [chunks][2]: pages to move, places
  int32_t* ranks;   // [n_pages]: among the pages to move or the places, -1
  int32_t keep, chunks, most;  // most: room for pairs
};

__global__ __launch_bounds__(kThreads) void compact_clear_kernel(u32x4* marks, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i < n) marks[i] = 0;
}

__global__ __launch_bounds__(kThreads) void compact_mark_kernel(CompactArgs a, int row_blocks) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (int(blockIdx.x) >= row_blocks) {
    const int64_t threads = int64_t(gridDim.x - row_blocks) * gridDim.y * kThreads;
    const int32_t count = min(max(a.count[0], 0), a.r.n_pages);
    for (int64_t i = ((int64_t(blockIdx.x) - row_blocks) * gridDim.y + blockIdx.y) * kThreads + threadIdx.x; i < count;
         i += threads) {
      const int32_t p = a.free_pages[i];
      if (p >= 0 && p < a.r.n_pages) a.idle[p] = 1;
    }
    return;
  }
  for (int64_t n = int64_t(blockIdx.x) * kWaves + wave; n < a.r.N; n += int64_t(row_blocks) * kWaves) {
    const int32_t* const row = a.r.table + n * a.r.width;
    const int32_t have = pages_of(a.r, a.held[n]);
    for (int64_t j0 = int64_t(blockIdx.y) * kSlice; j0 < have; j0 += int64_t(gridDim.y) * kSlice)
      for (int64_t j = j0 + lane; j < min(j0 + kSlice, int64_t(have)); j += 64) {
        const int32_t p = row[j];
        if (p >= 0 && p < a.r.n_pages) a.used[p] = 1;
      }
  }
}

// This thread's pages to move and places among its kEach, as bits.
struct Marks {
  uint32_t go, to;
};
__device__ __forceinline__ Marks marks_of(const CompactArgs& a, int64_t p0) {
  Marks m = {0, 0};
  const uint64_t used = *reinterpret_cast<const uint64_t*>(a.used + p0), idle = *reinterpret_cast<const uint64_t*>(a.idle + p0);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const bool u = used >> (8 * k) & 1, f = idle >> (8 * k) & 1, behind = p0 + k >= a.keep;
    m.go |= uint32_t(u && behind) << k;
    m.to |= uint32_t(f && !u && !behind) << k;
  }
  return m;
}

__global__ __launch_bounds__(kThreads) void compact_count_kernel(CompactArgs a) {
  __shared__ int32_t part[kWaves];
  const Marks m = marks_of(a, (int64_t(blockIdx.x) * kThreads + threadIdx.x) * kEach);
  const int32_t go = block_sum(__popc(m.go), part), to = block_sum(__popc(m.to), part);
  if (threadIdx.x == 0) a.counts[2 * blockIdx.x] = go, a.counts[2 * blockIdx.x + 1] = to;
}

__global__ __launch_bounds__(kThreads) void compact_rank_kernel(CompactArgs a) {
  __shared__ int32_t part[kWaves];
  const int tid = threadIdx.x;
  int32_t go_all = 0, to_all = 0, go = 0, to = 0;
  for (int c = tid; c < a.chunks; c += kThreads) {
    const int32_t g = a.counts[2 * c], t = a.counts[2 * c + 1];
    go_all += g;
    to_all += t;
    if (c < int(blockIdx.x)) go += g, to += t;
  }
  go_all = block_sum(go_all, part);
  to_all = block_sum(to_all, part);
  go = block_sum(go, part);
  to = block_sum(to, part);
  const int32_t moves = min(go_all, to_all);
  const int64_t p0 = (int64_t(blockIdx.x) * kThreads + tid) * kEach;
  const Marks m = marks_of(a, p0);
  int32_t total;
  go += block_inclusive(__popc(m.go), part, total) - __popc(m.go);
  to += block_inclusive(__popc(m.to), part, total) - __popc(m.to);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int64_t p = p0 + k;
    if (p >= a.r.n_pages) break;
    int32_t rank = -1;
    if (m.go >> k & 1) {
      rank = go++;
      if (rank < moves) a.pairs[2 * int64_t(rank)] = int32_t(p);
    } else if (m.to >> k & 1) {
      rank = to++;
      if (rank < moves) a.pairs[2 * int64_t(rank) + 1] = int32_t(p);
      else a.free_out[to_all - 1 - rank] = int32_t(p);
    }
    a.ranks[p] = rank;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.count_out[0] = to_all - moves;
    a.n_pairs[0] = moves;
    a.unmoved[0] = go_all - moves;
  }
}

__global__ __launch_bounds__(kThreads) void compact_apply_kernel(CompactArgs a) {
  const int64_t threads = int64_t(gridDim.x) * kThreads, first = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int32_t moves = a.n_pairs[0], left = a.count_out[0];
  for (int64_t i = first; i < int64_t(a.r.N) * a.r.width; i += threads) {
    const int32_t p = a.r.table[i];
    const int64_t n = i / a.r.width;
    int32_t to = p;
    if (p >= a.keep && p < a.r.n_pages && i - n * a.r.width < pages_of(a.r, a.held[n])) {
      const int32_t rank = a.ranks[p];
      if (rank >= 0 && rank < moves) to = a.pairs[2 * int64_t(rank) + 1];
    }
    a.table_out[i] = to;
  }
  for (int64_t p = first; p < a.r.n_pages; p += threads) {
    const int32_t rank = a.ranks[p];
    const bool moved = rank >= 0 && rank < moves;
    a.shares_out[p] = !moved ? a.shares[p] : p >= a.keep ? 0 : a.shares[a.pairs[2 * int64_t(rank)]];
    if (p >= left) a.free_out[p] = -1;
    if (p >= moves && p < a.most) a.pairs[2 * p] = a.pairs[2 * p + 1] = -1;
  }
}

// Page number `rank` among the set bits: the word by its sum, then the bit.
__device__ __forceinline__ int32_t select(const uint32_t* bits, const int32_t* before, int words, int32_t rank) {
  int lo = 0, hi = words - 1;   // the last word whose sum is at most rank
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (before[mid] <= rank) lo = mid; else hi = mid - 1;
  }
  uint32_t left = bits[lo];
  for (int32_t skip = rank - before[lo]; skip > 0; --skip) left &= left - 1;
  return lo * 32 + __ffs(left) - 1;
}

constexpr int kCompactPages = 1 << 15, kCompactRows = 2048, kCompactEntries = 1 << 15;   // of the pool, of the table
constexpr int kCompactWords = kCompactPages / 32;
static_assert(kCompactWords <= kSmallThreads, "a thread sums up one word");

__global__ __launch_bounds__(kSmallThreads) void compact_small_kernel(CompactArgs a) {
  __shared__ uint32_t go[kCompactWords], to[kCompactWords];   // pages to move, places
  __shared__ int32_t go_before[kCompactWords], to_before[kCompactWords];
  __shared__ int32_t have[kCompactRows];   // pages of a row
  __shared__ int32_t part[kSmallThreads / 64];
  const int tid = threadIdx.x, words = (a.r.n_pages + 31) / 32, entries = a.r.N * a.r.width;
  for (int w = tid; w < words; w += kSmallThreads) go[w] = to[w] = 0;
  for (int n = tid; n < a.r.N; n += kSmallThreads) have[n] = pages_of(a.r, a.held[n]);
  __syncthreads();
  const int32_t listed = min(max(a.count[0], 0), a.r.n_pages);
  for (int i = tid; i < listed; i += kSmallThreads) {
    const int32_t p = a.free_pages[i];
    if (p >= 0 && p < a.r.n_pages) atomicOr(to + p / 32, 1u << (p % 32));
  }
  constexpr int kAhead = 4;
  for (int i0 = tid; i0 < entries; i0 += kAhead * kSmallThreads) {
    int32_t page[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) page[k] = a.r.table[min(i0 + k * kSmallThreads, entries - 1)];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * kSmallThreads, n = i / a.r.width;
      if (i < entries && i - n * a.r.width < have[n] && page[k] >= 0 && page[k] < a.r.n_pages)
        atomicOr(go + page[k] / 32, 1u << (page[k] % 32));
    }
  }
  __syncthreads();
  int32_t go_mine = 0, to_mine = 0, go_all, to_all;
  if (tid < words) {
    const uint32_t behind = bits_from(tid, a.keep), used = go[tid];
    to[tid] &= ~used & ~behind;
    go[tid] = used & behind;
    go_mine = __popc(go[tid]);
    to_mine = __popc(to[tid]);
  }
  const int32_t go_upto = block_inclusive<kSmallThreads>(go_mine, part, go_all);
  const int32_t to_upto = block_inclusive<kSmallThreads>(to_mine, part, to_all);
  if (tid < words) {
    go_before[tid] = go_upto - go_mine;
    to_before[tid] = to_upto - to_mine;
  }
  __syncthreads();
  const int32_t moves = min(go_all, to_all), left = to_all - moves;
  const int threads = gridDim.x * kSmallThreads, start = blockIdx.x * kSmallThreads + tid;
  auto rank_of = [](const uint32_t* bits, const int32_t* before, int32_t p) {
    return before[p / 32] + __popc(bits[p / 32] & ((1u << (p % 32)) - 1));
  };
  auto marked = [](const uint32_t* bits, int32_t p) { return bits[p / 32] >> (p % 32) & 1; };
  for (int i = start; i < entries; i += threads) {
    const int n = i / a.r.width;
    int32_t p = a.r.table[i];
    if (p >= a.keep && p < a.r.n_pages && i - n * a.r.width < have[n]) {   // so it is marked
      const int32_t rank = rank_of(go, go_before, p);
      if (rank < moves) p = select(to, to_before, words, rank);
    }
    a.table_out[i] = p;
  }
  for (int32_t p = start; p < a.r.n_pages; p += threads) {
    int32_t shares = a.shares[p];
    if (marked(go, p)) {
      const int32_t rank = rank_of(go, go_before, p);
      if (rank < moves) {
        a.pairs[2 * rank] = p;
        shares = 0;
      }
    } else if (marked(to, p)) {
      const int32_t rank = rank_of(to, to_before, p);
      if (rank < moves) {
        a.pairs[2 * rank + 1] = p;
        shares = a.shares[select(go, go_before, words, rank)];
      } else {
        a.free_out[to_all - 1 - rank] = p;
      }
    }
    a.shares_out[p] = shares;
    if (p >= left) a.free_out[p] = -1;
    if (p >= moves && p < a.most) a.pairs[2 * p] = a.pairs[2 * p + 1] = -1;
  }
  if (start == 0) {
    a.count_out[0] = left;
    a.n_pairs[0] = moves;
    a.unmoved[0] = go_all - moves;
  }
}

// ---- copy ----
//
// Bound by HBM: a workgroup copies pieces of up to kPieceBytes of one page of one
// array, 16 bytes a thread and load, all loads of a piece before its stores. 96 MB
// of pages of 34 KB: 32 us (5.9 TB/s of reads and writes; 40 where the caches were
// not touched before).
constexpr int kLoads = 4, kPieceBytes = kThreads * 16 * kLoads;

struct CopyArgs {
  const int32_t* pairs;
  const int32_t* count;
  int64_t max_pairs;
  int32_t n_pages, n_arrays, pieces;  // pieces: of a page, all arrays
  u32x4* arrays[RGLRU_PAGE_COPY_ARRAYS];
  int32_t words[RGLRU_PAGE_COPY_ARRAYS];  // 16 bytes each
  int32_t ends[RGLRU_PAGE_COPY_ARRAYS];   // pieces up to this array's last
};

__global__ __launch_bounds__(kThreads) void copy_kernel(CopyArgs a) {
  const int64_t pairs = a.count == nullptr ? a.max_pairs : min(max(int64_t(a.count[0]), int64_t(0)), a.max_pairs);
  for (int64_t i = blockIdx.x; i < pairs * a.pieces; i += gridDim.x) {
    const int64_t pair = i / a.pieces;
    const int32_t piece = int32_t(i - pair * a.pieces);
    const int32_t from = a.pairs[2 * pair], to = a.pairs[2 * pair + 1];
    if (from < 0 || to < 0 || from >= a.n_pages || to >= a.n_pages || from == to) continue;
    int x = 0;
    while (piece >= a.ends[x]) ++x;
    const int32_t words = a.words[x], w0 = (piece - (x > 0 ? a.ends[x - 1] : 0)) * (kThreads * kLoads) + threadIdx.x;
    const u32x4* const src = a.arrays[x] + int64_t(from) * words;
    u32x4* const dst = a.arrays[x] + int64_t(to) * words;
    u32x4 v[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (w0 + k * kThreads < words) v[k] = src[w0 + k * kThreads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (w0 + k * kThreads < words) dst[w0 + k * kThreads] = v[k];
  }
}

bool valid(const rglru_paged_shape_t& s) { return valid_pages(s) && valid_table(s); }

Rows rows_of(const rglru_paged_shape_t& s, const int32_t* table) {
  return {table, int32_t(s.n_pages), s.n_seqs, s.max_pages, log2_of(s.page_size)};
}

template <size_t n>
bool aligned4(const void* const (&all)[n]) {
  for (const void* p : all)
    if (!aligned_to(p, 4)) return false;
  return true;
}
template <size_t n>
bool any_null(const void* const (&all)[n]) {
  for (const void* p : all)
    if (p == nullptr) return true;
  return false;
}

int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }
int64_t most(int64_t a, int64_t b) { return a > b ? a : b; }

// A wave per row, up to 1024 workgroups, and a row of workgroups per slice of the longest row.
dim3 row_grid(const rglru_paged_shape_t& s) {
  const int64_t x = least(ceil_div(s.n_seqs, kWaves), 1024);
  return dim3(unsigned(x), unsigned(least(ceil_div(s.max_pages, kSlice), most(2048 / x, 1))));
}

// Pools that one launch takes: every launch costs the host 2.6 us, but one workgroup (free) or each one (compact) passes over all
// bits of the pool. us on the GPU (replayed from a graph) and of a call among others, one launch and several:
//            rows, entries, pages     GPU               call
//   free     64, 1000, 600            6.9 and 7.6       10.4 and 15.5
//            64, 16 000, 8000         11.3 and 9.9      11.2 and 15.4
//            128, 16 000, 8000        11.9 and 9.1      11.9 and 15.1
//            64, 32 000, 16 000       16.4 and 11.7     16.3 and 15.2
//            64, 1000, 131 000        44 and 8.8        44 and 15
//   compact  64, 1000, 600            5.7 and 12.8      14.9 and 24.4
//            64, 32 000, 32 000       16.8 and 15.8     17.1 and 25.4
//            2000, 32 000, 32 000     17.4 and 14.7     17.8 and 25.3
//            64, 1000, 61 000         16.5 and 14.7     16.7 and 24
//            64, 1000, 131 000        28 and 15.5       29 and 24
// The bounds are where one launch starts to lose more than a fifth on the GPU; up to there a call costs 4 to 10 us less.
bool small(const rglru_paged_shape_t& s, int64_t pages, int rows, int64_t entries) {
  return s.n_pages <= pages && s.n_seqs <= rows && int64_t(s.n_seqs) * s.max_pages <= entries;
}
bool small_free(const rglru_paged_shape_t& s) { return small(s, kFreePages, kFreeRows, kFreeEntries); }
bool small_compact(const rglru_paged_shape_t& s) { return small(s, kCompactPages, kCompactRows, kCompactEntries); }

size_t free_bytes(const rglru_paged_shape_t& s) { return round_up(size_t(ceil_div(s.n_pages, kChunk)) * 4, 16); }

// Offsets of the workspace of compact: the marks, the chunks' counts, the ranks.
struct CompactSpace {
  size_t marks, counts, ranks, bytes;
  explicit CompactSpace(const rglru_paged_shape_t& s) {
    const size_t chunks = size_t(ceil_div(s.n_pages, kChunk));
    marks = chunks * kChunk;   // of one kind
    counts = 2 * marks;
    ranks = counts + round_up(chunks * 8, 16);
    bytes = ranks + round_up(size_t(s.n_pages) * 4, 16);
  }
};

}  // namespace
}  // namespace paged
}  // namespace rglru

using namespace rglru;

extern "C" rglru_status_t rglru_page_fork(const rglru_paged_shape_t* sp, const int32_t* fork_from, const int32_t* lens,
                                          const int32_t* held_lens, int32_t* block_table, int32_t* shares,
                                          const int32_t* free_pages, const int32_t* free_count, int32_t* pairs,
                                          int32_t* lens_out, int32_t* held_lens_out, int32_t* free_count_out,
                                          int32_t* unserved, void* stream) {
  if (sp == nullptr) return RGLRU_ERR_INVALID_ARGUMENT;
  const rglru_paged_shape_t s = *sp;
  const void* const all[] = {fork_from, lens,     block_table,   shares,         free_pages, free_count,
                             pairs,     lens_out, held_lens_out, free_count_out, unserved};
  if (!paged::valid(s) || paged::any_null(all)) return RGLRU_ERR_INVALID_ARGUMENT;
  if (!paged::aligned4(all) || !aligned_to(held_lens, 4)) return RGLRU_ERR_MISALIGNED;
  const int64_t seqs = int64_t(s.n_seqs) * 4;
  const paged::Bytes outs[] = {{block_table, seqs * s.max_pages}, {shares, s.n_pages * 4}, {pairs, 2 * seqs}, {lens_out, seqs},
                               {held_lens_out, seqs},             {free_count_out, 4},     {unserved, 4}};
  const paged::Bytes ins[] = {{fork_from, seqs}, {lens, seqs}, {held_lens, seqs}, {free_pages, s.n_pages * 4}, {free_count, 4}};
  if (paged::outputs_overlap(outs, ins)) return RGLRU_ERR_INVALID_ARGUMENT;
  paged::ForkArgs a;
  a.r = paged::rows_of(s, block_table);
  a.from = fork_from;
  a.lens = lens;
  a.held = held_lens != nullptr ? held_lens : lens;
  a.free_pages = free_pages;
  a.count = free_count;
  a.table = block_table;
  a.shares = shares;
  a.pairs = pairs;
  a.lens_out = lens_out;
  a.held_out = held_lens_out;
  a.count_out = free_count_out;
  a.unserved = unserved;
  const int64_t grid = paged::least(ceil_div(s.n_seqs, paged::kWaves), 1024);
  a.rows = int32_t(ceil_div(s.n_seqs, grid));
  paged::fork_kernel<<<unsigned(ceil_div(s.n_seqs, a.rows)), paged::kThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
  return launch_status();
}

extern "C" size_t rglru_page_free_workspace_bytes(const rglru_paged_shape_t* sp) {
  return sp == nullptr || !paged::valid(*sp) ? 0 : paged::free_bytes(*sp);
}

extern "C" rglru_status_t rglru_page_free(const rglru_paged_shape_t* sp, const int32_t* keep_lens, const int32_t* held_lens,
                                          const int32_t* block_table, int32_t* shares, int32_t* free_pages,
                                          const int32_t* free_count, int32_t* held_lens_out, int32_t* free_count_out,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  if (sp == nullptr) return RGLRU_ERR_INVALID_ARGUMENT;
  const rglru_paged_shape_t s = *sp;
  const void* const all[] = {keep_lens,  held_lens,     block_table,    shares,   free_pages,
                             free_count, held_lens_out, free_count_out, workspace};
  if (!paged::valid(s) || paged::any_null(all)) return RGLRU_ERR_INVALID_ARGUMENT;
  if (!paged::aligned4(all) || !aligned_to(workspace, 16)) return RGLRU_ERR_MISALIGNED;
  const size_t need = paged::free_bytes(s);
  if (workspace_bytes < need) return RGLRU_ERR_WORKSPACE_TOO_SMALL;
  const int64_t seqs = int64_t(s.n_seqs) * 4, pool = s.n_pages * 4;
  const paged::Bytes outs[] = {{shares, pool}, {free_pages, pool}, {held_lens_out, seqs}, {free_count_out, 4},
                               {workspace, int64_t(need)}};
  const paged::Bytes ins[] = {{keep_lens, seqs}, {held_lens, seqs}, {block_table, seqs * s.max_pages}, {free_count, 4}};
  if (paged::outputs_overlap(outs, ins)) return RGLRU_ERR_INVALID_ARGUMENT;
  paged::FreeArgs a;
  a.r = paged::rows_of(s, block_table);
  a.keep = keep_lens;
  a.held = held_lens;
  a.count = free_count;
  a.shares = shares;
  a.free_pages = free_pages;
  a.held_out = held_lens_out;
  a.count_out = free_count_out;
  a.counts = static_cast<int32_t*>(workspace);
  a.chunks = int32_t(ceil_div(s.n_pages, paged::kChunk));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (paged::small_free(s)) {
    paged::free_small_kernel<<<1, paged::kSmallThreads, 0, st>>>(a);
    return launch_status();
  }
  paged::free_mark_kernel<<<paged::row_grid(s), paged::kThreads, 0, st>>>(a);
  paged::free_count_kernel<<<unsigned(a.chunks), paged::kThreads, 0, st>>>(a);
  paged::free_list_kernel<<<unsigned(a.chunks), paged::kThreads, 0, st>>>(a);
  return launch_status();
}

extern "C" size_t rglru_page_compact_workspace_bytes(const rglru_paged_shape_t* sp) {
  return sp == nullptr || !paged::valid(*sp) ? 0 : paged::CompactSpace(*sp).bytes;
}

extern "C" rglru_status_t rglru_page_compact(const rglru_paged_shape_t* sp, int64_t keep_pages, const int32_t* held_lens,
                                             const int32_t* block_table, const int32_t* shares, const int32_t* free_pages,
                                             const int32_t* free_count, int32_t* block_table_out, int32_t* shares_out,
                                             int32_t* free_pages_out, int32_t* free_count_out, int32_t* pairs,
                                             int32_t* n_pairs, int32_t* unmoved, void* workspace, size_t workspace_bytes,
                                             void* stream) {
  if (sp == nullptr) return RGLRU_ERR_INVALID_ARGUMENT;
  const rglru_paged_shape_t s = *sp;
  const void* const all[] = {held_lens,  block_table,    shares,         free_pages, free_count, block_table_out,
                             shares_out, free_pages_out, free_count_out, n_pairs,    unmoved,    workspace};
  if (!paged::valid(s) || keep_pages < 0 || keep_pages > s.n_pages || paged::any_null(all)) return RGLRU_ERR_INVALID_ARGUMENT;
  const int64_t room = paged::least(keep_pages, s.n_pages - keep_pages);
  if (room > 0 && pairs == nullptr) return RGLRU_ERR_INVALID_ARGUMENT;
  if (!paged::aligned4(all) || !aligned_to(pairs, 4) || !aligned_to(workspace, 16)) return RGLRU_ERR_MISALIGNED;
  const paged::CompactSpace space(s);
  if (workspace_bytes < space.bytes) return RGLRU_ERR_WORKSPACE_TOO_SMALL;
  const int64_t seqs = int64_t(s.n_seqs) * 4, table = seqs * s.max_pages, pool = s.n_pages * 4;
  const paged::Bytes outs[] = {{block_table_out, table}, {shares_out, pool}, {free_pages_out, pool}, {free_count_out, 4},
                               {pairs, 8 * room},        {n_pairs, 4},       {unmoved, 4},           {workspace, int64_t(space.bytes)}};
  const paged::Bytes ins[] = {{held_lens, seqs}, {block_table, table}, {shares, pool}, {free_pages, pool}, {free_count, 4}};
  if (paged::outputs_overlap(outs, ins)) return RGLRU_ERR_INVALID_ARGUMENT;
  uint8_t* const at = static_cast<uint8_t*>(workspace);
  paged::CompactArgs a;
  a.r = paged::rows_of(s, block_table);
  a.held = held_lens;
  a.shares = shares;
  a.free_pages = free_pages;
  a.count = free_count;
  a.table_out = block_table_out;
  a.shares_out = shares_out;
  a.free_out = free_pages_out;
  a.count_out = free_count_out;
  a.pairs = pairs;
  a.n_pairs = n_pairs;
  a.unmoved = unmoved;
  a.used = at;
  a.idle = at + space.marks;
  a.counts = reinterpret_cast<int32_t*>(at + space.counts);
  a.ranks = reinterpret_cast<int32_t*>(at + space.ranks);
  a.keep = int32_t(keep_pages);
  a.chunks = int32_t(ceil_div(s.n_pages, paged::kChunk));
  a.most = int32_t(room);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (paged::small_compact(s)) {
    const int64_t all = paged::most(int64_t(s.n_seqs) * s.max_pages, s.n_pages);
    paged::compact_small_kernel<<<unsigned(ceil_div(all, paged::kSmallThreads)), paged::kSmallThreads, 0, st>>>(a);
    return launch_status();
  }
  const int64_t words = int64_t(space.counts) / 16;
  paged::compact_clear_kernel<<<unsigned(ceil_div(words, paged::kThreads)), paged::kThreads, 0, st>>>(
      reinterpret_cast<paged::u32x4*>(at), words);
  dim3 grid = paged::row_grid(s);
  const int row_blocks = int(grid.x);
  grid.x += unsigned(paged::least(ceil_div(s.n_pages, paged::kThreads), 1024));
  paged::compact_mark_kernel<<<grid, paged::kThreads, 0, st>>>(a, row_blocks);
  paged::compact_count_kernel<<<unsigned(a.chunks), paged::kThreads, 0, st>>>(a);
  paged::compact_rank_kernel<<<unsigned(a.chunks), paged::kThreads, 0, st>>>(a);
  const int64_t entries = paged::most(int64_t(s.n_seqs) * s.max_pages, s.n_pages);
  paged::compact_apply_kernel<<<unsigned(paged::least(ceil_div(entries, paged::kThreads), 2048)), paged::kThreads, 0, st>>>(a);
  return launch_status();
}

extern "C" rglru_status_t rglru_page_copy(int64_t n_pages, const int32_t* pairs, int64_t max_pairs, const int32_t* count,
                                          int32_t n_arrays, void* const* arrays, const int64_t* page_bytes, void* stream) {
  constexpr int64_t kMost = int64_t(1) << 31;
  if (n_pages < 1 || n_pages >= kMost || max_pairs < 0 || max_pairs >= kMost || n_arrays < 1 ||
      n_arrays > RGLRU_PAGE_COPY_ARRAYS || arrays == nullptr || page_bytes == nullptr || (max_pairs > 0 && pairs == nullptr))
    return RGLRU_ERR_INVALID_ARGUMENT;
  paged::CopyArgs a;
  a.pairs = pairs;
  a.count = count;
  a.max_pairs = max_pairs;
  a.n_pages = int32_t(n_pages);
  a.n_arrays = n_arrays;
  a.pieces = 0;
  int64_t bytes = 0;
  for (int x = 0; x < n_arrays; ++x) {
    if (arrays[x] == nullptr || page_bytes[x] < 16 || page_bytes[x] >= kMost || page_bytes[x] % 16 != 0)
      return RGLRU_ERR_INVALID_ARGUMENT;
    bytes += page_bytes[x];
    a.arrays[x] = static_cast<paged::u32x4*>(arrays[x]);
    a.words[x] = int32_t(page_bytes[x] / 16);
    a.pieces += int32_t(ceil_div(page_bytes[x], paged::kPieceBytes));
    a.ends[x] = a.pieces;
  }
  if (bytes >= kMost) return RGLRU_ERR_INVALID_ARGUMENT;
  bool aligned = aligned_to(pairs, 4) && aligned_to(count, 4);
  for (int x = 0; x < n_arrays; ++x) aligned = aligned && aligned_to(arrays[x], 16);
  if (!aligned) return RGLRU_ERR_MISALIGNED;
  const paged::Bytes ins[] = {{pairs, 8 * max_pairs}, {count, 4}};
  for (int x = 0; x < n_arrays; ++x)
    for (int y = 0; y <= x; ++y) {
      // against the inputs (y = x), or an earlier array
      const paged::Bytes one[] = {{arrays[x], n_pages * page_bytes[x]}};
      const paged::Bytes other[] = {{arrays[y], n_pages * page_bytes[y]}};
      if (y == x ? paged::outputs_overlap(one, ins) : paged::outputs_overlap(one, other)) return RGLRU_ERR_INVALID_ARGUMENT;
    }
  if (max_pairs == 0) return RGLRU_OK;
  const int64_t grid = max_pairs >= 4096 || max_pairs * a.pieces >= 4096 ? 4096 : max_pairs * a.pieces;
  paged::copy_kernel<<<unsigned(grid), paged::kThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
  return launch_status();
}
