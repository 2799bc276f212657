// Attention of new tokens over a paged key/value cache in bf16 or float32 (include/paged_attn.h).
//
// The mathematics, the kernel for many rows and what joins the pieces stand in paged_attn_core.h; here are the kernel for few
// rows and the entry points.
#include <hip/hip_runtime.h>

#include "paged_attn_core.h"

namespace rglru {
namespace paged {

namespace {

// ---- few rows: at most 32 per unit (decode steps, drafts) ----
//
// Bound by the bytes of the cache: a unit of r rows does 4 r D flops for
// every 4 D bytes (bf16) of keys and values, 16 flops per byte at 16 rows where
// the card has some 250. Each wave streams tiles of 32 keys of its own
// through its own LDS buffers without a barrier; the waves of a workgroup merge
// at the end of a unit. What counts is how many bytes are in flight: a
// wave asks for the next keys (values) as soon as it has read the buffer that
// they go to. 64 sequences of up to 8192 keys, 8 key heads of 128 in bf16: 0.195
// ms, 5.5 TB/s; of 32 768 keys: 6.1 TB/s.
constexpr int kNarrowKeys = 32, kNarrowOver = 6;

// In a call that needs the wide kernel it takes the sequences of few rows too where there are at most kFewSeqs sequences and
// kFewUnits (sequence of few rows, key head) pairs: it saves a launch, but works through such a unit as slowly as through
// one of many rows. 618 calls of a chunk of 200 or 1000 tokens and 1 to 15 single tokens, all after 200 to 8000 tokens, 1
// to 16 key heads, timed with the wide kernel alone and with both: taking the better of the two by this rule costs 1.6 %
// more than by the clock in bf16 at D = 64 and 2.2 to 2.8 % in float32 (without the second bound 5 and 7 to 13 %), 0.2 %
// in bf16 at D = 128 and 256, whose best bound is past what was measured (240). A chunk of 1000 after 2000 at D = 128, 4
// key heads, alone and both: beside 15 single tokens 56 and 60 us, in float32 273 and 239; beside 47 87 and 78.
template <typename E, int D>
constexpr int kFewUnits = sizeof(E) == 4 ? 24 : D == 64 ? 64 : 256;

template <typename E, int D>
struct Narrow {
  static constexpr int kTileBytes = kNarrowKeys * D * int(sizeof(E));
  // 128 KB of LDS per CU, four waves in a workgroup. Up to 8 KB a tile each wave has two buffers of keys and two of
  // values (and there are two workgroups at 4 KB), at 16 KB one of each, at 32 KB one for both. kGroups also tells
  // the compiler how many waves share a SIMD: with two it keeps the output out of the accumulation registers, which it
  // copies to and fro otherwise (D = 64: 22.4 -> 21 us for 16 sequences of 2000 keys).
  static constexpr int kWaves = 4, kStretches = 1;
  static constexpr int kBuffers = kTileBytes <= 8192 ? 4 : 32768 / kTileBytes;
  static constexpr int kGroups = kTileBytes == 4096 ? 2 : 1;
  static constexpr int kThreads = kWaves * 64;
  // The one buffer holds four slices of columns, each loaded anew as soon as it is read: those of the values take the
  // place of those of the keys and the other way round. Half of the queries lie in LDS, as the registers would not hold
  // them and the output (float32, D = 256, 64 sequences of 8000 keys, 2 key heads: whole tiles in turn 3.9 TB/s, slices
  // 4.4, with half of the queries in LDS 5.1, now that no register spills 5.7).
  static constexpr int kSlice = kBuffers == 1 ? D / 4 : D;
};

// Length of a unit of a sequence in the line.
__device__ __forceinline__ int32_t narrow_size(const AttnArgs& a, const Seq& s) {
  if (s.fresh == 0 || int64_t(s.fresh) * a.group > kNarrowRows) return 0;
  const Span x = span_of<kNarrowKeys>(a, s, 0, s.fresh * a.group - 1);
  return x.hi - x.lo + kNarrowOver;
}

// ---- few rows: the kernel ----
template <typename E, int D>
__global__ __launch_bounds__((Narrow<E, D>::kThreads), (Narrow<E, D>::kGroups)) void narrow_kernel(AttnArgs a) {
  using P = Narrow<E, D>;
  constexpr int kLoads = P::kTileBytes / 1024;
  using W = Wave<E, D, P::kSlice>;
  __shared__ __align__(1024) unsigned char buf[P::kWaves * P::kBuffers * P::kTileBytes + W::kRestBytes];
  __shared__ int64_t scan_part[P::kWaves];
  __shared__ Seq found;
  __shared__ int32_t found_seq;
  __shared__ int64_t found_rest;
  __shared__ float merge_c[P::kWaves][32], merge_l[P::kWaves][32];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = blockIdx.x;
  if (b == a.narrow.grid) {
    list_row_tiles<Wide<E, D>, P::kThreads>(a, scan_part, a.sched, a.row_tiles, a.sched + 2 + a.max_tiles);
    return;
  }

  // Total length, then the sequence that holds this stretch's start. Up to a sequence per thread both come of one scan.
  Seq own = {0, 0, 0};
  int64_t total = 0, size = 0, upto = 0;
  for (int n0 = 0; n0 < a.N; n0 += P::kThreads) {
    int64_t sum;
    own = {0, 0, 0};
    if (n0 + tid < a.N) own = seq_of(a, n0 + tid);
    size = int64_t(narrow_size(a, own)) * a.Hkv;
    upto = block_scan<P::kThreads>(size, scan_part, sum);
    total += sum;
  }
  if (tid == 0) a.narrow.joins[4 * b + 2] = 0;
  if (total == 0) return;
  const Line line(total, a.narrow.grid, P::kWaves);
  int64_t pos = line.start(b);
  const int64_t end = line.start(b + 1);
  if (pos >= end) return;
  int64_t found_before = 0;
  for (int n0 = 0;; n0 += P::kThreads) {
    int64_t sum = total;
    if (a.N > P::kThreads) {
      own = {0, 0, 0};
      if (n0 + tid < a.N) own = seq_of(a, n0 + tid);
      size = int64_t(narrow_size(a, own)) * a.Hkv;
      upto = found_before + block_scan<P::kThreads>(size, scan_part, sum);
    }
    if (pos >= upto - size && pos < upto) {
      found = own;
      found_seq = n0 + tid;
      found_rest = pos - (upto - size);
    }
    found_before += sum;
    if (pos < found_before || n0 + P::kThreads >= a.N) break;
  }
  __syncthreads();
  int n = __builtin_amdgcn_readfirstlane(found_seq);
  int64_t rest = found_rest;   // position within the sequence's units
  Seq s = {__builtin_amdgcn_readfirstlane(found.start), __builtin_amdgcn_readfirstlane(found.fresh),
           __builtin_amdgcn_readfirstlane(found.kv)};
  W w;
  w.rest = (lds_u8*)buf + P::kWaves * P::kBuffers * P::kTileBytes;
  lds_u8* const mine = (lds_u8*)buf + wave * P::kBuffers * P::kTileBytes;
  while (pos < end && n < a.N) {
    const int32_t rows = int64_t(s.fresh) * a.group > kNarrowRows ? 0 : s.fresh * a.group;
    if (rows == 0) {
      if (++n < a.N) s = seq_of(a, n);
      continue;
    }
    const Span x = span_of<kNarrowKeys>(a, s, 0, rows - 1);
    const int32_t tiles = x.hi - x.lo, size = tiles + kNarrowOver;
    const int hk = __builtin_amdgcn_readfirstlane(int(rest / size));
    const int32_t in = int32_t(rest - int64_t(hk) * size);   // where this stretch enters the unit and leaves it
    const int32_t out = int32_t(min(int64_t(size), in + (end - pos)));
    if (out <= kNarrowOver) break;   // left to the next workgroup
    const int32_t t0 = max(in - kNarrowOver, 0), t1 = out - kNarrowOver;
    const_i32* row = (const_i32*)(a.table + int64_t(n) * a.width);
    const int32_t last_page = max((s.kv - 1) >> a.lps, 0);
    w.queries(a, s, hk, lane & 31, rows, lane);
    w.start(a, s, lane & 31, rows);
    if constexpr (W::kRestBytes > 0) {
#pragma unroll
      for (int i = 0; i < D / 16 - W::kHeld; ++i)
        if (i % P::kWaves == wave) w.put_query(i, lane);
      __syncthreads();
    }

    constexpr int kSegs = kNarrowKeys / kSeg, kSegLoads = kLoads / kSegs;
    // the pages of the tile to load next are looked up one tile ahead
    int32_t pages[kSegs];
    int64_t at[kSegs];
    auto look_up = [&](int32_t t) {
      const int32_t kv0 = __builtin_amdgcn_readfirstlane((x.lo + t) * kNarrowKeys);
#pragma unroll
      for (int i = 0; i < kSegs; ++i) pages[i] = seg_page(a, row, last_page, kv0 + i * kSeg);
    };
    auto locate = [&](int32_t t) {
      const int32_t kv0 = __builtin_amdgcn_readfirstlane((x.lo + t) * kNarrowKeys);
#pragma unroll
      for (int i = 0; i < kSegs; ++i) at[i] = seg_offset<E, D>(a, pages[i], hk, kv0 + i * kSeg);
    };
    // mine: the buffers of keys, then those of values
    constexpr int kW = P::kWaves, kTwo = P::kBuffers == 4;
    const uint32_t keys_at = uint32_t(uintptr_t(mine));
    look_up(t0 + wave);
    wait_loads<0>();   // no store of the unit before is counted below
    if constexpr (P::kBuffers > 1) {
      auto load_keys = [&](int32_t t, uint32_t to) {
        locate(t);
#pragma unroll
        for (int i = 0; i < kSegs; ++i)
          load_rows<E, D, false, kSegLoads>(a.kc + at[i], i * kSeg, to + i * kSegLoads * 1024, lane);
      };
      auto load_values = [&](uint32_t to) {
#pragma unroll
        for (int i = 0; i < kSegs; ++i)
          load_rows<E, D, true, kSegLoads>(a.vc + at[i], i * kSeg, to + i * kSegLoads * 1024, lane);
      };
      constexpr int kValues = P::kBuffers / 2 * P::kTileBytes;
      const uint32_t values_at = keys_at + kValues;
      uint32_t half = 0;
#pragma unroll 1
      for (int i = 0; i < 1 + kTwo; ++i)
        if (t0 + wave + i * kW < t1) {
          load_keys(t0 + wave + i * kW, keys_at + i * P::kTileBytes);
          load_values(values_at + i * P::kTileBytes);
          look_up(t0 + wave + (i + 1) * kW);
        }
      for (int32_t t = t0 + wave; t < t1; t += kW) {
        const bool next = t + kW < t1;                // a further tile
        const bool after = t + (1 + kTwo) * kW < t1;  // and one for the buffers that this tile leaves
        const int32_t kv0 = (x.lo + t) * kNarrowKeys;
        const bool full = kv0 + kNarrowKeys - 1 <= x.first && (a.window == 0 || kv0 > x.last - a.window);
        Frag<E> p[kNarrowKeys / 16];
        // behind these keys are in flight: these values and, of two buffers, the next tile
        if (kTwo && next) wait_loads<3 * kLoads>();
        else wait_loads<kLoads>();
        w.template scores<kNarrowKeys>(a, mine + half, kv0, full, lane, p, [&](int) {
          if (after) {
            wait_reads();
            load_keys(t + (1 + kTwo) * kW, keys_at + half);
          }
        });
        // behind these values: the keys just asked for and, of two buffers, the next tile
        if (kTwo && after) wait_loads<3 * kLoads>();
        else if (kTwo && next) wait_loads<2 * kLoads>();
        else if (!kTwo && after) wait_loads<kLoads>();
        else wait_loads<0>();
        lds_u8* const vt = mine + kValues + half;
        if (!full && __any(any_odd<E, P::kTileBytes, 64>(vt, lane))) {
          w.template mark<kNarrowKeys>(vt, kv0, lane, 0);
          clean<E, P::kTileBytes, 64>(vt, lane);
        }
        w.template values<kNarrowKeys>(vt, p, lane);
        if (after) {
          wait_reads();
          load_values(values_at + half);
          look_up(t + (2 + kTwo) * kW);
        }
        if (kTwo) half ^= P::kTileBytes;
      }
    } else {
      constexpr int kSlices = D / P::kSlice, kSliceLoads = kLoads / kSlices, kSliceBytes = P::kTileBytes / kSlices;
      static_assert(kSlices == 4, "the waits below");
      auto load_keys = [&](int c) {
#pragma unroll
        for (int i = 0; i < kSegs; ++i)
          load_slice<E, D, P::kSlice, false>(a.kc + at[i], c, i * kSeg, keys_at + c * kSliceBytes + i * (kSliceBytes / kSegs), lane);
      };
      auto load_values = [&](int c) {
#pragma unroll
        for (int i = 0; i < kSegs; ++i)
          load_slice<E, D, P::kSlice, true>(a.vc + at[i], c, i * kSeg, keys_at + c * kSliceBytes + i * (kSliceBytes / kSegs), lane);
      };
      if (t0 + wave < t1) {
        locate(t0 + wave);
#pragma unroll
        for (int c = 0; c < kSlices; ++c) load_keys(c);
        look_up(t0 + wave + kW);
      }
      for (int32_t t = t0 + wave; t < t1; t += kW) {
        const bool next = t + kW < t1;
        const int32_t kv0 = (x.lo + t) * kNarrowKeys;
        const bool full = kv0 + kNarrowKeys - 1 <= x.first && (a.window == 0 || kv0 > x.last - a.window);
        Frag<E> p[kNarrowKeys / 16];
        // A slice is waited for when the one before it has not quite been read: behind it are in flight the later ones
        // and those that took the place of the earlier ones but for the last, two in all; behind the first, three.
        w.template scores<kNarrowKeys>(
            a, mine, kv0, full, lane, p,
            [&](int c) {
              wait_reads();
              load_values(c);
            },
            [&](int c) {
              if (c == 0) wait_loads<3 * kSliceLoads>();
              else wait_loads<2 * kSliceLoads>();
            });
        if (next) {
          locate(t + kW);
          look_up(t + 2 * kW);
        }
        w.template values<kNarrowKeys>(
            mine, p, lane,
            [&](int c) {
              if (c == 0) wait_loads<3 * kSliceLoads>();
              else if (c == 1 || next) wait_loads<2 * kSliceLoads>();
              else if (c == 2) wait_loads<kSliceLoads>();
              else wait_loads<0>();
              lds_u8* const vt = mine + c * kSliceBytes;
              if (!full && __any(any_odd<E, kSliceBytes, 64>(vt, lane))) {
                w.template mark<kNarrowKeys>(mine, kv0, lane, c);
                clean<E, kSliceBytes, 64>(vt, lane);
              }
            },
            [&](int c) {
              if (!next) return;
              wait_reads();
              load_keys(c);
            });
      }
    }

    // The waves merge: maxima and sums first, then every thread sums some columns over the waves.
    const float l_all = w.finish();
    __syncthreads();   // the buffers are free
    float* const sums = reinterpret_cast<float*>(buf);
    const int q = lane & 31, h = lane >> 5;
    if (h == 0) {
      merge_c[wave][q] = w.c;
      merge_l[wave][q] = l_all;
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == tiles;
    float* const part = a.narrow.parts + int64_t(2 * b + (t0 == 0 ? 1 : 0)) * part_floats<D>(kNarrowRows);
    // half of the columns at a time, in the buffers of the tiles
#pragma unroll
    for (int x0 = 0; x0 < D / 32; x0 += (D / 32 + 1) / 2) {
      constexpr int kX = (D / 32 + 1) / 2, kC = kX * 32, kRow = kC + 4;  // 4 floats against bank conflicts
      static_assert(P::kWaves * 32 * kRow * 4 <= int(sizeof(buf)), "merge buffer");
      if (q < rows) {
#pragma unroll
        for (int y = 0; y < kX; ++y)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const f32x16& v = w.o[x0 + y];
            float4 f = {v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
            *reinterpret_cast<float4*>(sums + (wave * 32 + q) * kRow + y * 32 + 8 * r + 4 * h) = f;
          }
      }
      __syncthreads();
      for (int e = tid; e < rows * (kC / 4); e += P::kThreads) {
        const int qq = e / (kC / 4), d = (e % (kC / 4)) * 4;
        float top = -INFINITY;
        for (int v = 0; v < P::kWaves; ++v) top = fmaxf(top, merge_c[v][qq]);
        const float base = top == -INFINITY ? 0.0f : top;
        float4 acc = {0, 0, 0, 0};
        float l = 0.0f;
        for (int v = 0; v < P::kWaves; ++v) {
          const float f = __builtin_amdgcn_exp2f(merge_c[v][qq] - base);
          const float4 z = *reinterpret_cast<const float4*>(sums + (v * 32 + qq) * kRow + d);
          // a part without weights counts too, by a factor of 0: what it saw may not have been finite
          acc.x += f * z.x;
          acc.y += f * z.y;
          acc.z += f * z.z;
          acc.w += f * z.w;
          l += f * merge_l[v][qq];
        }
        const int col = x0 * 32 + d;
        if (whole) {
          const float inv = top == -INFINITY ? 0.0f : 1.0f / l;
          if (top == -INFINITY) acc = {0, 0, 0, 0};
          const int64_t r = out_row(a, s, hk, qq);
          store4<E>(a.o + (r * D + col) * sizeof(E), acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
          if (a.lse != nullptr && col == 0) a.lse[r] = top == -INFINITY ? -INFINITY : (top + log2f(l)) * kLn2;
        } else {
          *reinterpret_cast<float4*>(part + qq * D + col) = acc;
          if (col == 0) {
            part[kNarrowRows * D + qq] = top;
            part[kNarrowRows * (D + 1) + qq] = l;
          }
        }
      }
      __syncthreads();
    }
    if (tid == 0 && t0 > 0 && line.start(b - 1) <= pos - in + kNarrowOver) {
      // the first cut of this unit: the one before is not within it
      a.narrow.joins[4 * b] = n;
      a.narrow.joins[4 * b + 1] = hk;
      a.narrow.joins[4 * b + 3] = 0;
      a.narrow.joins[4 * b + 2] = int32_t(1 + line.before(pos - in + size) - b);
    }
    pos += out - in;
    rest = out < size ? rest + (out - in) : (hk + 1 < a.Hkv ? int64_t(hk + 1) * size : 0);
    if (out == size && hk + 1 == a.Hkv && ++n < a.N) s = seq_of(a, n);
  }
}

// 32 sequences of 4096 keys, 32 rows on each of 4 key heads of 128: the narrow kernel alone takes 60 us, the wide one 65.
template <typename E, int D>
Plan plan_of(const rglru_paged_shape_t& s) {
  return plan_of<Narrow<E, D>, Wide<E, D>, D>(s, kNarrowKeys, kFewUnits<E, D>);
}

template <typename E, int D>
size_t bytes_of(const rglru_paged_shape_t& s) {
  return plan_of<E, D>(s).bytes;
}

template <typename E, int D>
void launch(const rglru_paged_shape_t& s, AttnArgs a, uint8_t* workspace, hipStream_t st) {
  using W = Wide<E, D>;
  const Plan p = plan_of<E, D>(s);
  lay_out(a, p, workspace);
  if (p.narrow) narrow_kernel<E, D><<<unsigned(p.narrow_grid + p.wide), Narrow<E, D>::kThreads, 0, st>>>(a);
  if (p.wide) {
    if (!p.narrow && !p.own_list) sched_kernel<W><<<1, kSchedThreads, 0, st>>>(a);
    wide_kernel<E, D><<<unsigned(p.wide_grid), W::kThreads, 0, st>>>(a);
  }
  join<E, D, W>(s, a, p, st);
}

}  // namespace
}  // namespace paged
}  // namespace rglru

using namespace rglru;

extern "C" size_t rglru_paged_attn_workspace_bytes(const rglru_paged_shape_t* sp) {
  if (sp == nullptr || paged::check(*sp) != RGLRU_OK) return 0;
  return RGLRU_PAGED_DISPATCH(*sp, paged::bytes_of, *sp);
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
  const size_t need = rglru_paged_attn_workspace_bytes(&s);
  if (workspace_bytes < need) return RGLRU_ERR_WORKSPACE_TOO_SMALL;
  const int64_t dense = int64_t(s.q_heads) * s.head_dim, seqs = int64_t(s.n_seqs) * 4;
  const int64_t cache = s.n_pages * s.page_size * s.kv_heads * s.head_dim * esize;
  const paged::Bytes outs[] = {{o, s.n_tokens * dense * esize}, {lse, s.n_tokens * s.q_heads * 4}, {workspace, int64_t(need)}};
  const paged::Bytes ins[] = {{cu_seqlens, seqs + 4}, {kv_lens, seqs},  {block_table, seqs * s.max_pages},
                              {q, paged::rows_size(s.n_tokens, stride, dense, esize)}, {k_cache, cache}, {v_cache, cache}};
  if (paged::outputs_overlap(outs, ins)) return RGLRU_ERR_INVALID_ARGUMENT;
  paged::AttnArgs a;
  paged::set_args(a, s, cu_seqlens, kv_lens, block_table, q, k_cache, v_cache, o, lse);
  RGLRU_PAGED_DISPATCH(s, paged::launch, s, a, static_cast<uint8_t*>(workspace), static_cast<hipStream_t>(stream));
  return launch_status();
}
