// Attention of new tokens over a paged key/value cache: what the kernels of every kind of cache share.
//
// Mathematics. A row is one (token, query head); the rows of a key head are
// (token, head of its group) pairs in that order, so a group's heads share the
// keys and values that a workgroup reads. A wave holds 32 rows as the columns
// of S^T = K Q^T (32x32 MFMA): a lane owns one row, so the running maximum and
// sum of the softmax are per-lane scalars and the sum over keys needs no
// exchange but one between the two half-waves for the maximum. The
// accumulator layout of S^T (keys 4h..4h+3 and 8+4h..8+4h+3 of every 16 in
// half-wave h) is the operand layout of O^T = V^T P^T up to the order of the
// keys, and the sum over keys does not care for their order: the weights go
// from one product into the next without leaving their registers, and V^T is
// read out of row-major V with the transposing LDS read (4 keys of one column
// per lane). Scores, maxima, sums and outputs are float32; bf16 weights are
// rounded to bf16 where they enter the product (what the matrix cores take).
// The output is rescaled only where the maximum grew by more than 8 (log2):
// the weights stay below 2^8 then, which costs float32 and bf16 nothing, and
// most tiles skip the rescale.
//
// float32 uses the float32 MFMA with the same lane layouts, eight 2-deep
// products for one 16-deep one.
//
// What a row must not see must not reach it, infinities and NaN included:
// scores are replaced where they are masked, but a weight of 0 times an
// infinite value is NaN. The values of a tile that some row does not see in
// full are therefore looked at first; where one is not finite, products of 0/1
// operands mark the (row, column) pairs that see a +inf, a -inf or a NaN, and
// those values are replaced by 0 in LDS before the tile is worked on.
#pragma once

#include <hip/hip_runtime.h>

#include "paged_common.h"

namespace rglru {
namespace paged {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) unsigned char lds_u8;
typedef __attribute__((address_space(4))) const int32_t const_i32;  // read through the scalar cache

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;  // growth of the maximum (log2) that the weights absorb without a rescale

// An operand of a 32x32x16 product: 8 elements per lane (16 bytes of bf16, 32 of float32).
template <typename E>
struct Frag;
template <>
struct Frag<uint16_t> {
  static constexpr uint32_t kSigns = 0x80008000u;
  u32x4 w;
};
template <>
struct Frag<float> {
  static constexpr uint32_t kSigns = 0x80000000u;
  u32x8 w;
};

__device__ __forceinline__ f32x16 mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.w), __builtin_bit_cast(bf16x8, b.w), c, 0,
                                                 0, 0);
}
__device__ __forceinline__ f32x16 mma(const Frag<float>& a, const Frag<float>& b, f32x16 c) {
  const f32x8 x = __builtin_bit_cast(f32x8, a.w), y = __builtin_bit_cast(f32x8, b.w);
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[j], y[j], c, 0, 0, 0);
  return c;
}

// float32 against a tile in bf16: three bf16 parts, each what is left of the one before cut to 8 bits, so that they hold all
// 24 bits.
struct Split {
  static constexpr uint32_t kSigns = 0x80008000u;
  u32x4 w[3];
};
__device__ __forceinline__ f32x16 mma(const Frag<uint16_t>& a, const Split& b, f32x16 c) {
#pragma unroll
  for (int j = 2; j >= 0; --j)
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.w), __builtin_bit_cast(bf16x8, b.w[j]), c, 0,
                                                0, 0);
  return c;
}

// What queries and weights in E are beside keys and values of type C in LDS.
template <typename E, typename C>
struct Operand {
  typedef Frag<E> type;
};
template <>
struct Operand<float, uint16_t> {
  typedef Split type;
};

// All bits cleared that are not in `keep`, those in `flip` changed.
template <typename E>
__device__ __forceinline__ void set_bits(Frag<E>& f, uint32_t keep, uint32_t flip) {
  f.w = (f.w & keep) ^ flip;
}
__device__ __forceinline__ void set_bits(Split& f, uint32_t keep, uint32_t flip) {
#pragma unroll
  for (int j = 0; j < 3; ++j) f.w[j] = (f.w[j] & keep) ^ flip;
}

__device__ __forceinline__ Frag<uint16_t> pack(const float* p, uint16_t) {
  Frag<uint16_t> f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f.w[j] = f32x2_to_bf16x2(p[2 * j], p[2 * j + 1]);
  return f;
}
__device__ __forceinline__ Frag<float> pack(const float* p, float) {
  Frag<float> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.w[j] = __float_as_uint(p[j]);
  return f;
}

// The next part of two floats, which become what is left.
__device__ __forceinline__ uint32_t split_off(float& a, float& b) {
  const uint32_t x = __float_as_uint(a) & 0xFFFF0000u, y = __float_as_uint(b) & 0xFFFF0000u;
  a -= __uint_as_float(x);
  b -= __uint_as_float(y);
  return x >> 16 | y;
}
__device__ __forceinline__ Split split(const float* p) {
  Split f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = p[2 * j], b = p[2 * j + 1];
#pragma unroll
    for (int i = 0; i < 3; ++i) f.w[i][j] = split_off(a, b);
  }
  return f;
}
// Queries may be infinite: a part that is left of one is 0, not NaN.
__device__ __forceinline__ Split split_query(const u32x4& lo, const u32x4& hi) {
  float p[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = __uint_as_float(lo[j]), p[4 + j] = __uint_as_float(hi[j]);
  Split f = split(p);
#pragma unroll
  for (int i = 1; i < 3; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t keep = (fabsf(p[2 * j]) < INFINITY ? 0xFFFFu : 0u) | (fabsf(p[2 * j + 1]) < INFINITY ? 0xFFFF0000u : 0u);
      f.w[i][j] &= keep;
    }
#pragma unroll
  for (int j = 0; j < 8; ++j)   // a NaN whose first 8 bits are those of an infinity
    if (p[j] != p[j]) f.w[0][j / 2] |= 0x40u << (16 * (j & 1));
  return f;
}
template <typename O, typename E>
__device__ __forceinline__ O pack_as(const float* p) {
  if constexpr (sizeof(O) == sizeof(Split)) return split(p);
  else return pack(p, E{});
}

// The elements of a word that are not finite (bf16 pairs or a float), all their bits set.
__device__ __forceinline__ uint32_t odd_bits(uint32_t w, uint16_t) {
  const uint32_t top = (((w & 0x7F807F80u) + 0x00800080u) >> 15) & 0x00010001u;
  return (top << 16) - top;
}
__device__ __forceinline__ uint32_t odd_bits(uint32_t w, float) {
  return (w & 0x7F800000u) == 0x7F800000u ? ~0u : 0u;
}

// The same as a test: the top bits of what this returns.
__device__ __forceinline__ uint32_t odd_carry(uint32_t w, uint16_t) { return (w & 0x7F807F80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t odd_carry(uint32_t w, float) { return (w & 0x7F800000u) + 0x00800000u; }

// A 0/1 operand that marks +inf and NaN (sign 0) or -inf and NaN (sign 1).
__device__ __forceinline__ Frag<uint16_t> marks(const Frag<uint16_t>& f, uint32_t sign) {
  Frag<uint16_t> m;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w = 0;
#pragma unroll
    for (int s = 0; s < 32; s += 16) {
      const uint32_t x = (f.w[j] >> s) & 0xFFFFu;
      const bool nan = (x & 0x7FFFu) > 0x7F80u;
      w |= (nan || x == (sign << 15 | 0x7F80u) ? 0x3F80u : 0u) << s;
    }
    m.w[j] = w;
  }
  return m;
}
__device__ __forceinline__ Frag<float> marks(const Frag<float>& f, uint32_t sign) {
  Frag<float> m;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool nan = (f.w[j] & 0x7FFFFFFFu) > 0x7F800000u;
    m.w[j] = nan || f.w[j] == (sign << 31 | 0x7F800000u) ? 0x3F800000u : 0u;
  }
  return m;
}

__device__ __forceinline__ float half_max(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A tile of kRows rows of the cache in LDS, in pieces of 16 bytes. The piece
// at column c of row r lies at column c ^ swizzle(r), chosen so that the 16
// lanes that one LDS cycle serves fall on different banks: keys are read 16
// bytes per lane down a column of rows, values 4 rows x 64 bytes at a time
// (bf16, transposing) or a row of floats per half-wave (float32). The
// swizzles are linear over XOR, so what depends on the instruction and on the
// lane separates.
template <typename E, int D>
struct Tile {
  static constexpr int kRowBytes = D * int(sizeof(E));
  static constexpr int kCols = kRowBytes / 16;          // pieces of a row
  static constexpr int kLoadRows = 64 / kCols;          // rows that one load of a wave fetches
  __device__ static constexpr int swz_k(int r) { return kCols == 8 ? (r >> 1) & 7 : r & 15; }
  __device__ static constexpr int swz_v(int r) {
    return sizeof(E) == 4 ? ((r >> 2) & 1) << 3 : kCols == 8 ? ((r >> 1) & 1) << 2 : (r & 3) << 2;
  }
};

// What one kernel leaves for the join.
struct Cuts {
  int32_t* joins;  // [grid][4]: sequence, key head, pieces (0: none) and first row of what the cut before stretch b parted; or
                   // [N * Hkv][2], by unit: pieces (0: none) and the stretch that the first cut is before
  float* parts;    // [grid][2]: partial results of a stretch's first and last unit
  int32_t grid;    // stretches
};

struct RowTile;

struct AttnArgs {
  const int32_t* cu;
  const int32_t* kv_lens;
  const int32_t* table;
  const uint8_t* q;
  const uint8_t* kc;
  const uint8_t* vc;
  uint8_t* o;
  float* lse;
  int64_t* sched;   // the row tiles of the wide kernel (see list_row_tiles)
  RowTile* row_tiles;
  Cuts narrow, wide;
  int64_t q_stride;
  int32_t T, n_pages, N, width, lps, Hq, Hkv, group, window, max_tiles;
  int32_t own_list;    // the wide kernel's workgroups list the row tiles themselves
  int32_t least_rows;  // the wide kernel's sequences have more rows than this
  float scale2;     // |scale| log2 e (1 for a scale of 0, whose queries are zeroed)
  int32_t q_sign;   // sign of the scale: -1, 0, 1
};

// One sequence's lengths, clamped so that whatever is stored every access stays in bounds.
struct Seq {
  int32_t start, fresh, kv;
};
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int n) {
  Seq s;
  s.start = min(max(a.cu[n], 0), a.T);
  s.fresh = min(max(a.cu[n + 1], s.start), a.T) - s.start;
  s.kv = min(max(a.kv_lens[n], 0), a.width << a.lps);
  return s;
}

// Positions of rows r0 .. r1 (inclusive) of a sequence, -1 before its start, and the tiles of kv that they see.
struct Span {
  int32_t first, last;  // positions
  int32_t lo, hi;       // tiles [lo, hi), at least one
};
template <int BN>
__device__ __forceinline__ Span span_of(const AttnArgs& a, const Seq& s, int32_t r0, int32_t r1) {
  Span x;
  x.first = max(s.kv - s.fresh + r0 / a.group, -1);
  x.last = max(s.kv - s.fresh + r1 / a.group, -1);
  x.lo = a.window > 0 ? max(x.first - a.window + 1, 0) / BN : 0;
  x.hi = max((x.last + BN) / BN, x.lo + 1);
  return x;
}

// Eight rows of the cache lie in one page (the smallest page), so they are one
// piece of memory. seg_page looks up the page of rows j .. j + 7 of a sequence,
// seg_offset gives their place, in bytes.
constexpr int kSeg = 8;

__device__ __forceinline__ int32_t seg_page(const AttnArgs& a, const_i32* row, int32_t last_page, int32_t j) {
  return row[min(j >> a.lps, last_page)];
}
template <typename E, int D>
__device__ __forceinline__ int64_t seg_offset(const AttnArgs& a, int32_t page, int hk, int32_t j) {
  const int64_t p = min(max(page, 0), a.n_pages - 1);
  return (((p * a.Hkv + hk) << a.lps) + (j & ((1 << a.lps) - 1))) * Tile<E, D>::kRowBytes;
}

// 64 lanes x 16 bytes from base + off + kAt to LDS at `to` + kAt. Written out
// because the compiler, which cannot tell the buffers apart, would wait for every
// load in flight before each transposing LDS read. It has no output register; its arrival
// is waited for by wait_loads, which every path passes before the tile is read.
template <int kAt>
__device__ __forceinline__ void load_lds(uint32_t to, uint32_t off, const uint8_t* base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 offset:%3" ::"s"(to), "v"(off), "s"(base),
               "n"(kAt)
               : "memory");
}

// Loads kCount KB of consecutive rows, from row r of a tile on, straight into LDS (`to`: where row r goes).
template <typename E, int D, bool kValues, int kCount, int kFrom = 0>
__device__ __forceinline__ void load_rows(const uint8_t* base, int r, uint32_t to, int lane) {
  using L = Tile<E, D>;
  if constexpr (kFrom < kCount) {
    const int x = lane / L::kCols, c = lane % L::kCols;
    const int lane_swz = kValues ? L::swz_v(x) : L::swz_k(x);
    const int row = r + kFrom * L::kLoadRows;
    const int load_swz = kValues ? L::swz_v(row) : L::swz_k(row);
    const uint32_t off = uint32_t((((c ^ lane_swz) * 16) ^ (load_swz * 16)) + x * L::kRowBytes);
    load_lds<(kFrom % 4) * 1024>(to + (kFrom & ~3) * 1024, off, base + (kFrom & ~3) * 1024);
    load_rows<E, D, kValues, kCount, kFrom + 1>(base, r, to, lane);
  }
}

// The same for 8 rows of slice `c` of a tile that lies in slices of kSlice columns: rows r .. r + 7, kept kRowBytes apart.
template <typename E, int D, int kSlice, bool kValues>
__device__ __forceinline__ void load_slice(const uint8_t* base, int c, int r, uint32_t to, int lane) {
  using L = Tile<E, kSlice>;
  const int x = lane / L::kCols, col = lane % L::kCols;
  const int lane_swz = kValues ? L::swz_v(x) : L::swz_k(x);
#pragma unroll
  for (int i = 0; i < kSeg / L::kLoadRows; ++i) {
    const int row = r + i * L::kLoadRows;
    const int load_swz = kValues ? L::swz_v(row) : L::swz_k(row);
    const uint32_t off = uint32_t((((col ^ lane_swz) * 16) ^ (load_swz * 16)) + x * Tile<E, D>::kRowBytes);
    load_lds<0>(to + i * 1024, off, base + c * L::kRowBytes + i * L::kLoadRows * Tile<E, D>::kRowBytes);
  }
}

// Waits until at most kMost vector memory operations of this wave are in flight (63 where that is more than can be said).
template <int kMost>
__device__ __forceinline__ void wait_loads() {
  constexpr int n = kMost < 63 ? kMost : 63;
  __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | ((n >> 4) << 14));
  asm volatile("" ::: "memory");
}

// Hides where a value comes from: what is computed of it is computed here, and not kept in registers across tiles.
__device__ __forceinline__ void fresh_value(int& x) { asm volatile("" : "+v"(x)); }

// Keeps the compiler from moving anything across: left to itself it saves registers by putting every LDS read right
// before its product and waits for each.
__device__ __forceinline__ void order() { __builtin_amdgcn_sched_barrier(0); }

// Waits until this wave's LDS reads have returned, before their place is loaded anew.
__device__ __forceinline__ void wait_reads() {
  __builtin_amdgcn_s_waitcnt(0xC07F);
  asm volatile("" ::: "memory");
}

struct Nothing {
  __device__ __forceinline__ void operator()(int) const {}
};

// 32 rows of one wave. A tile may lie in LDS as slices of kSlice columns, each laid out like a tile of that width, so
// that one slice is fetched into while others are read.
template <typename E, int D, int kSlice = D, typename C = E>
struct Wave {
  using L = Tile<C, kSlice>;
  using O = typename Operand<E, C>::type;
  static constexpr int kSlices = D / kSlice;
  static constexpr int kHeld = kSlices > 1 ? D / 32 : D / 16;  // operands of queries in registers; the others in LDS, at `rest`
  static constexpr int kRestBytes = (D / 16 - kHeld) * 64 * int(sizeof(O));
  lds_u8* rest;
  O q[D / 16];
  f32x16 o[D / 32];
  float m, c, l;     // running maximum of the scores, the same times scale2 (log2 units), sum of the weights (this half-wave's keys)
  int32_t lo, hi;    // the keys this lane's row sees: lo <= j <= hi

  // Loads this lane's share of the queries of row r.
  __device__ __forceinline__ void queries(const AttnArgs& a, const Seq& s, int hk, int32_t r, int32_t rows, int lane) {
    const bool live = r < rows;
    const int32_t t = live ? r / a.group : 0, g = live ? r - t * a.group : 0;
    const uint8_t* src = a.q + ((s.start + t) * a.q_stride + int64_t(hk * a.group + g) * D) * sizeof(E);
    const int h = lane >> 5;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      if constexpr (sizeof(O) == sizeof(Split)) q[x].w[0] = q[x].w[1] = q[x].w[2] = 0;
      else q[x].w = 0;
      if (live) {
        // in pieces of 16 bytes, which is what the rows are aligned to
        const u32x4* const from = reinterpret_cast<const u32x4*>(src + (x * 16 + h * 8) * sizeof(E));
        if constexpr (sizeof(O) == sizeof(Split)) q[x] = split_query(from[0], from[1]);
        else if constexpr (sizeof(E) == 2) q[x].w = from[0];
        else q[x].w = __builtin_shufflevector(from[0], from[1], 0, 1, 2, 3, 4, 5, 6, 7);
      }
    }
  }

  __device__ __forceinline__ void start(const AttnArgs& a, const Seq& s, int32_t r, int32_t rows) {
    if (a.q_sign <= 0) {
      const uint32_t keep = a.q_sign == 0 ? 0u : ~0u, flip = a.q_sign < 0 ? O::kSigns : 0u;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) set_bits(q[x], keep, flip);
    }
#pragma unroll
    for (int x = 0; x < D / 32; ++x) o[x] = 0.0f;
    m = c = -INFINITY;
    l = 0.0f;
    hi = r < rows ? max(s.kv - s.fresh + r / a.group, -1) : -1;
    lo = a.window > 0 ? max(hi - a.window + 1, 0) : 0;
  }

  // Operand kHeld + i of the queries, kept in LDS in pieces of 16 bytes a lane.
  __device__ __forceinline__ void put_query(int i, int lane) {
    auto* const to = (__attribute__((address_space(3))) u32x4*)(rest + i * 64 * int(sizeof(O)));
#pragma unroll
    for (int j = 0; j < int(sizeof(O)) / 16; ++j)
      to[j * 64 + lane] = reinterpret_cast<const u32x4*>(&q[kHeld + i])[j];
  }
  __device__ __forceinline__ O get_query(int i, int lane) const {
    O f;
    const auto* const from = (const __attribute__((address_space(3))) u32x4*)(rest + i * 64 * int(sizeof(O)));
#pragma unroll
    for (int j = 0; j < int(sizeof(O)) / 16; ++j) reinterpret_cast<u32x4*>(&f)[j] = from[j * 64 + lane];
    return f;
  }

  // The sum over both half-waves. A row whose scores are all NaN has no maximum: it gets one, so that it is not taken
  // for a row that sees nothing.
  __device__ __forceinline__ float finish() {
    const float sum = half_sum(l);
    if (sum != sum && c == -INFINITY) c = 0.0f;
    return sum;
  }

  // Weights of BN keys from kv0 on; `full`: every row of the wave sees them all. done(c) is called when the reads of
  // slice c have been issued, and its last product; of several slices ready(c) before its first read.
  template <int BN, typename Done, typename Ready = Nothing>
  __device__ __forceinline__ void scores(const AttnArgs& a, const lds_u8* kt, int32_t kv0, bool full, int lane,
                                         O* p, Done done, Ready ready = {}) {
    const int h = lane >> 5;
    f32x16 s[BN / 32];
    {
      // product i: keys of subtile i / (D / 16), elements 16 (i % (D / 16)) on; operands are read kAhead products early
      constexpr int kSteps = D / 16, kAll = BN / 32 * kSteps, kAhead = sizeof(C) == 2 ? 4 : 2;
      constexpr int kOne = kSteps / kSlices;
      static_assert(kSlices == 1 || (BN == 32 && kAhead < kOne), "a slice's products follow each other");
      const int r = lane & 31;
      int at = r * L::kRowBytes + (sizeof(C) == 2 ? (h ^ L::swz_k(r)) * 16 : ((2 * h) ^ L::swz_k(r)) * 16);
      fresh_value(at);
      Frag<C> k[kAhead];
      O z[kAhead];
      auto fetch = [&](int i) {
        const int b = i / kSteps, x = i % kOne;
        const lds_u8* p = kt + (b + i % kSteps / kOne) * 32 * L::kRowBytes;
        if (kSlices > 1 && x == 0) ready(i / kOne);
        if (i % kSteps >= kHeld) z[i % kAhead] = get_query(i % kSteps - kHeld, lane);
        if constexpr (sizeof(C) == 2) {
          k[i % kAhead].w = *(const __attribute__((address_space(3))) u32x4*)(p + (at ^ (x * 32)));
        } else {
          const u32x4 w0 = *(const __attribute__((address_space(3))) u32x4*)(p + (at ^ (x * 64)));
          const u32x4 w1 = *(const __attribute__((address_space(3))) u32x4*)(p + (at ^ (x * 64 + 16)));
          k[i % kAhead].w = __builtin_shufflevector(w0, w1, 0, 1, 2, 3, 4, 5, 6, 7);
        }
      };
#pragma unroll
      for (int b = 0; b < BN / 32; ++b) s[b] = 0.0f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(i);
#pragma unroll
      for (int i = 0; i < kAll; ++i) {
        const int b = i / kSteps, x = i % kSteps;
        s[b] = mma(k[i % kAhead], x < kHeld ? q[x] : z[i % kAhead], s[b]);
        if (kSlices > 1 && i % kOne == kOne - 1) done(i / kOne);
        if (i + kAhead < kAll) fetch(i + kAhead);
        order();
      }
    }
    if (kSlices == 1) done(0);
    if (!full) {
#pragma unroll
      for (int b = 0; b < BN / 32; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int32_t j = kv0 + b * 32 + 8 * (r / 4) + r % 4 + 4 * h;
          if (j < lo || j > hi) s[b][r] = -INFINITY;
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < BN / 32; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
    top = half_max(top);
    // the wave branches together, each row decides for itself: what other rows see must not change its bits
    const bool grow = top * a.scale2 > c + kSlack;
    if (__any(grow)) {
      const float m_new = grow ? fmaxf(m, top) : m, c_new = m_new * a.scale2;
      // 0 below 2^-126: a finite output leaves nothing then, an infinite one stays (this tile's marks may be among them).
      // Rows that had no maximum have nothing to rescale, so a unit's first tile skips it (few rows at D = 256 17.4 -> 15.8 us).
      const float keep = grow && c != -INFINITY ? __builtin_amdgcn_exp2f(c - c_new) : 1.0f;
      if (__any(keep != 1.0f)) {
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[x][r] = fabsf(o[x][r]) == INFINITY ? o[x][r] : o[x][r] * keep;
      }
      l *= keep;
      m = m_new;
      c = grow ? c_new : c;
    }
    const float base = c == -INFINITY ? 0.0f : c;
    float sum = 0.0f;
#pragma unroll
    for (int b = 0; b < BN / 32; ++b)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float w[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          w[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][8 * y + r], a.scale2, -base));
          sum += w[r];
        }
        p[2 * b + y] = pack_as<O, E>(w);
      }
    l += sum;
  }

  // Adds BN weighted values to the output; ready(c) and done(c) as above, of several slices.
  template <int BN, typename Ready = Nothing, typename Done = Nothing>
  __device__ __forceinline__ void values(const lds_u8* vt, const O* p, int lane, Ready ready = {}, Done done = {}) {
    constexpr int kSteps = BN / 16, kAll = D / 32 * kSteps, kAhead = sizeof(C) == 2 ? 4 : 2, kOne = kAll / kSlices;
    static_assert(kSlices == 1 || kAhead < kOne, "a slice's products follow each other");
    int start = value_at(lane);
    fresh_value(start);
    Frag<C> v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (kSlices > 1 && i == 0) ready(0);
      v[i] = value_frag<BN>(vt, i / kSteps, i % kSteps, start);
    }
#pragma unroll
    for (int i = 0; i < kAll; ++i) {
      o[i / kSteps] = mma(v[i % kAhead], p[i % kSteps], o[i / kSteps]);
      if (kSlices > 1 && i % kOne == kOne - 1) done(i / kOne);
      if (i + kAhead < kAll) {
        if (kSlices > 1 && (i + kAhead) % kOne == 0) ready((i + kAhead) / kOne);
        v[i % kAhead] = value_frag<BN>(vt, (i + kAhead) / kSteps, (i + kAhead) % kSteps, start);
      }
      order();
    }
  }

  // Where a lane's values start: bf16, row 4h + (lane % 16) / 4, columns 16 ((lane / 16) % 2) + 4 (lane % 4) .., of which the
  // transposing read hands the lane 4 rows of column lane % 32; float32, row 4h, column lane % 32.
  __device__ static __forceinline__ int value_at(int lane) {
    const int h = lane >> 5;
    if constexpr (sizeof(C) == 2) {
      const int r = 4 * h + (lane & 15) / 4, col = 2 * ((lane >> 4) & 1) + (lane & 3) / 2;
      return r * L::kRowBytes + (col ^ L::swz_v(r)) * 16 + (lane & 1) * 8;
    } else {
      const int r = 4 * h, col = lane & 31;
      return r * L::kRowBytes + ((col / 4) ^ L::swz_v(r)) * 16 + (col % 4) * 4;
    }
  }

  // The operand of columns 32 x .. and keys 16 y .. of a tile. 32 columns are 4 (8) pieces of a row, which the swizzle
  // takes to others of the row's pieces: an XOR.
  template <int BN>
  __device__ __forceinline__ Frag<C> value_frag(const lds_u8* vt, int x, int y, int start) const {
    Frag<C> v;
    constexpr int kCols = kSlice / 32;
    const int at = (start ^ (x % kCols * 32 * int(sizeof(C)))) + (x / kCols * BN + y * 16) * L::kRowBytes;
    if constexpr (sizeof(C) == 2) {
      const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(vt + at));
      const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(vt + at + 8 * L::kRowBytes));
      const u32x2 a = __builtin_bit_cast(u32x2, v0), b = __builtin_bit_cast(u32x2, v1);
      v.w = __builtin_shufflevector(a, b, 0, 1, 2, 3);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v.w[j] = *(const __attribute__((address_space(3))) uint32_t*)(vt + at + (8 * (j / 4) + j % 4) * L::kRowBytes);
    }
    return v;
  }

  // Marks what values that are not finite do to this wave's rows: a row that sees a +inf or a NaN gets +inf in its
  // column, one that sees a -inf or a NaN gets -inf (so NaN gives NaN). Products of 0/1 operands, which are finite.
  // The columns of slice c.
  template <int BN>
  __device__ __forceinline__ void mark(const lds_u8* vt, int32_t kv0, int lane, int c) {
    Frag<C> see[BN / 16];
#pragma unroll
    for (int y = 0; y < BN / 16; ++y) {
      float one[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int32_t j = kv0 + 16 * y + 8 * (r / 4) + r % 4 + 4 * (lane >> 5);
        one[r] = j >= lo && j <= hi ? 1.0f : 0.0f;
      }
      see[y] = pack(one, C{});
    }
#pragma unroll
    for (int x = c * (kSlice / 32); x < (c + 1) * (kSlice / 32); ++x)
#pragma unroll 1
      for (uint32_t sign = 0; sign < 2; ++sign) {
        f32x16 sum = 0.0f;
#pragma unroll
        for (int y = 0; y < BN / 16; ++y) sum = mma(marks(value_frag<BN>(vt, x, y, value_at(lane)), sign), see[y], sum);
#pragma unroll
        for (int r = 0; r < 16; ++r) o[x][r] += sum[r] > 0.0f ? (sign ? -INFINITY : INFINITY) : 0.0f;
      }
  }
};

// Whether this thread's share of a tile of values holds one that is not finite.
template <typename E, int kTileBytes, int kThreads>
__device__ __forceinline__ bool any_odd(const lds_u8* vt, int thread) {
  uint32_t odd = 0;
#pragma unroll
  for (int i = 0; i < kTileBytes; i += kThreads * 16) {
    const u32x4 w = *(const __attribute__((address_space(3))) u32x4*)(vt + i + thread * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) odd |= odd_carry(w[j], E{});
  }
  return (odd & Frag<E>::kSigns) != 0;
}

// Replaces them by 0.
template <typename E, int kTileBytes, int kThreads>
__device__ __forceinline__ void clean(lds_u8* vt, int thread) {
  for (int i = thread * 16; i < kTileBytes; i += kThreads * 16) {
    u32x4 w = *(const __attribute__((address_space(3))) u32x4*)(vt + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] &= ~odd_bits(w[j], E{});
    *(__attribute__((address_space(3))) u32x4*)(vt + i) = w;
  }
}

template <typename E>
__device__ __forceinline__ void store4(uint8_t* p, float a, float b, float c, float d) {
  if constexpr (sizeof(E) == 2) {
    u32x2 w = {f32x2_to_bf16x2(a, b), f32x2_to_bf16x2(c, d)};
    *reinterpret_cast<u32x2*>(p) = w;
  } else {
    u32x4 w = {__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d)};
    *reinterpret_cast<u32x4*>(p) = w;
  }
}

// The D outputs of one row times `f` (0 for a row without weights, whatever its sums are), 16 bytes per lane and
// instruction. The two half-waves hold 4 elements each of every 8: for bf16 they trade, so that one has the 8 of an even
// group and the other those of the next.
template <typename E, int D>
__device__ __forceinline__ void store_row(uint8_t* to, const f32x16* o, float f, int h) {
#pragma unroll
  for (int y = 0; y < D / 32; ++y)
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = f == 0.0f ? 0.0f : o[y][4 * k + j] * f;
      if constexpr (sizeof(E) == 2) {
        const auto a = __builtin_amdgcn_permlane32_swap(f32x2_to_bf16x2(e[0], e[1]), f32x2_to_bf16x2(e[4], e[5]), false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(f32x2_to_bf16x2(e[2], e[3]), f32x2_to_bf16x2(e[6], e[7]), false, false);
        const u32x4 w = {a[0], b[0], a[1], b[1]};
        *reinterpret_cast<u32x4*>(to + (y * 32 + 8 * (k + h)) * 2) = w;
      } else {
        store4<float>(to + (y * 32 + 8 * k + 4 * h) * 4, e[0], e[1], e[2], e[3]);
        store4<float>(to + (y * 32 + 8 * k + 8 + 4 * h) * 4, e[4], e[5], e[6], e[7]);
      }
    }
}

// Output row of (sequence, key head, row), as an index of [T, Hq].
__device__ __forceinline__ int64_t out_row(const AttnArgs& a, const Seq& s, int hk, int32_t r) {
  const int32_t t = r / a.group;
  return int64_t(s.start + t) * a.Hq + hk * a.group + (r - t * a.group);
}

// A value that all lanes share, for the compiler to know.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return int64_t(uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(v >> 32)))) << 32 |
                 uint32_t(__builtin_amdgcn_readfirstlane(int(v))));
}

// A partial result: kRows rows of D floats (not normalised), then kRows maxima (log2 units) and kRows sums.
template <int D>
constexpr int part_floats(int rows) {
  return rows * (D + 2);
}

// The share of the work of workgroup b: the units (sequence, key head, row
// tile) stand in one line, each as long as its tiles of keys and a fixed part for
// starting and ending it (kOver tiles' worth), and every workgroup takes an equal stretch of that line. A unit
// that lies in one stretch is finished there; the pieces of one that is cut
// go to `parts` (slot 0: the unit began in an earlier stretch, slot 1: it began
// here) and the join after the cut merges them in order, so the bits do not
// depend on timing. A cut within the fixed part moves to the unit's start.
struct Line {
  int64_t total;
  int32_t parts;  // stretches
  __device__ __forceinline__ Line(int64_t total_, int grid, int least) : total(total_) {
    parts = int(min(max(total / least, int64_t(1)), int64_t(grid)));
  }
  // Where stretch b starts.
  __device__ __forceinline__ int64_t start(int64_t b) const { return total * min(b, int64_t(parts)) / parts; }
  // Stretches that start before `at`.
  __device__ __forceinline__ int64_t before(int64_t at) const { return (at * parts + total - 1) / total; }
};

constexpr int kNarrowRows = 32;   // rows of a unit that the kernels for few rows take at most

// Row tiles that the wide kernel's workgroups list themselves, and sequences that a call without a kernel for few rows has at most.
constexpr int kFewSeqs = 16, kOwnTiles = 256;

template <int kThreads>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int d = 1; d < 64; d *= 2) {
    const int64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 63) part[wave] = v;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < wave) v += part[w];
    total += part[w];
  }
  return v;
}

// ---- many rows: chunks of a prompt, and whatever stands beside them in a batch ----
//
// Bound by the matrix cores. kRows rows of one (sequence, key head) share
// every tile of kKeys keys and values, which the waves fetch together into one
// of two LDS buffers while they work on the other; one barrier a tile. 2048
// tokens after 30 011, 32 query and 8 key heads of 128: 0.91 to 1.00 ms by card, 1.0 to 1.1
// PFLOP/s, where an 8192^3 library product reaches 1.14 on the same card; the
// matrix pipes are busy 54 % of the time at the 1.9 GHz that the power allows.
// Eight prompts of 4096 with a window of 2048, 10 heads of 256: 0.54 to 0.58 ms,
// 0.9 PFLOP/s.
template <typename E, int D, typename C = E>
struct Wide {
  static constexpr bool kBf16 = sizeof(E) == 2, kTiles16 = sizeof(C) == 2;
  // bf16: two waves per SIMD, so that one's softmax runs beside the other's products. float32 products take 16 times as
  // long, so less shows of the softmax: one wave per SIMD in a workgroup, half as many rows left idle
  static constexpr int kWaves = kBf16 ? 8 : 4;
  // Workgroups on a CU: two where the registers allow it (float32, D = 64), so that one's softmax runs beside the other's
  // products (2048 tokens after 8000, 4 key heads: 378 -> 337 us, 307 now), but one for calls whose stretches would be shorter than
  // kShort tiles. 208 calls of 1 to 20 chunks of 50 to 1000 tokens after 0 to 2000, 2 to 8 key heads, timed with one and with two:
  // one is up to 1.3 times as fast at 1 to 3 tiles, the same at 8 to 12, two 1.1 times as fast from 20 on.
  static constexpr int kGroups = !kBf16 && D == 64 ? 2 : 1, kShort = 10;
  static constexpr int kThreads = kWaves * 64;
  static constexpr int kRows = kWaves * 32;
  static constexpr int kKeys = D == 256 || !kBf16 ? 32 : 64;
  // What starting and ending a unit costs, in tiles: 15 us where a tile takes 1.6 (bf16, D = 256), 8 where it takes 1.9
  // (D = 128); float32 tiles take 16 times as long. At D = 64 126 calls (1 to 20 chunks of 100 to 2000 tokens after 0 to 4000,
  // with and without a window) take 0.6 % more in the mean with 3 and 0.7 % more with 8.
  // float32 on tiles of bf16: 3 (1 chunk of 2048 after 8000 137, 263, 468 us with 1 and 135, 265, 460 with 3 at D = 64, 128, 256).
  static constexpr int kOver = !kTiles16 ? 1 : !kBf16 ? 3 : D == 256 ? 9 : D == 128 ? 4 : 5;
  static constexpr int kTileBytes = kKeys * D * int(sizeof(C));
};

// The row tiles of all sequences: sched[0] their number, sched[1] the length
// of one key head's units, then for each tile the length before it, then for each its RowTile.
// One workgroup writes them: the narrow kernel's last, beside the others' work, or, where that kernel does not run, a
// launch of its own; up to kOwnTiles of them every workgroup of the wide kernel lists for itself, in LDS, which takes 2 us
// where the launch takes 6.
struct __attribute__((aligned(32))) RowTile {
  int32_t n, r0;               // sequence, first row
  int32_t start, fresh, kv;    // its lengths
  int32_t lo, hi;              // tiles of keys
  int32_t unused;
};
typedef __attribute__((address_space(4))) const RowTile const_row_tile;

template <typename W, int kThreads>
__device__ __forceinline__ void list_row_tiles(const AttnArgs& a, int64_t* part, int64_t* sched, RowTile* which,
                                               int64_t* starts) {
  constexpr int kRows = W::kRows, kKeys = W::kKeys, kOver = W::kOver;
  const int tid = threadIdx.x;
  int64_t* const before = sched + 2;   // `starts`: row tiles before each sequence
  int64_t count = 0, sum;
  for (int n0 = 0; n0 < a.N; n0 += kThreads) {
    const int n = n0 + tid;
    const int64_t rows = n < a.N ? int64_t(seq_of(a, n).fresh) * a.group : 0;
    const int64_t v = rows > a.least_rows ? (rows + kRows - 1) / kRows : 0;
    const int64_t inc = count + block_scan<kThreads>(v, part, sum);
    if (n < a.N) starts[n] = inc - v;
    count += sum;
  }
  count = min(count, int64_t(a.max_tiles));
  __syncthreads();
  int64_t total = 0;
  for (int64_t t0 = 0; t0 < count; t0 += kThreads) {
    const int64_t t = t0 + tid;
    int64_t v = 0;
    if (t < count) {
      int lo = 0, hi = a.N - 1;  // the last sequence that starts at or before t; empty ones share their start with the next
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (starts[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const Seq s = seq_of(a, lo);
      // first, last, second, last but one ..: under a causal mask the first see few keys and the last many, and in this
      // order stretches of one length are whole units more often
      const int32_t i = int32_t(t - starts[lo]), all = (s.fresh * a.group + kRows - 1) / kRows;
      const int32_t rt = i % 2 == 0 ? i / 2 : all - 1 - i / 2, r0 = rt * kRows;
      const Span x = span_of<kKeys>(a, s, r0, max(min(r0 + kRows, s.fresh * a.group) - 1, r0));
      v = x.hi - x.lo + kOver;
      which[t] = {lo, r0, s.start, s.fresh, s.kv, x.lo, x.hi, 0};
    }
    const int64_t inc = total + block_scan<kThreads>(v, part, sum);
    if (t < count) before[t] = inc - v;
    total += sum;
  }
  if (tid == 0) {
    sched[0] = count;
    sched[1] = total;
  }
}

constexpr int kSchedThreads = 1024;
constexpr int kCus = 256;   // of the card

template <typename W>
__global__ __launch_bounds__(kSchedThreads) void sched_kernel(AttnArgs a) {
  __shared__ int64_t part[kSchedThreads / 64];
  list_row_tiles<W, kSchedThreads>(a, part, a.sched, a.row_tiles, a.sched + 2 + a.max_tiles);
}

// Merges the pieces of every unit that was cut, in the order of the keys. A
// row takes D / 4 threads; the other threads of a workgroup take further rows
// or, where there are many pieces, further pieces of the same row.
constexpr int kJoinThreads = 256, kManyPieces = 64;

// Share y of `shares` of the rows from r0 on of one unit, whose second piece is that of stretch b; kCols columns from d0 on.
template <typename E, int D, int kCols = D>
__device__ __forceinline__ void join_unit(const AttnArgs& a, const Cuts& cuts, int kRows, int b, int pieces, int n, int hk, int r0,
                                          int y, int shares, int d0 = 0) {
  constexpr int kLanes = kCols / 4, kSets = kJoinThreads / kLanes, kAhead = 8, kShare = 16;
  __shared__ float4 acc_s[kSets][kLanes];
  __shared__ float l_s[kSets], c_s[kSets];
  const int tid = threadIdx.x;
  const Seq s = seq_of(a, n);
  const int64_t part_size = int64_t(kRows) * (D + 2);
  const int rows = min(kRows, s.fresh * a.group - r0);
  // The sets share a row's pieces where there are many and that takes fewer reads in a row than a set per row.
  const bool share = pieces > kShare && (rows + shares - 1) / shares * kAhead < pieces;
  const int set = tid / kLanes, d = d0 + (tid % kLanes) * 4;
  auto write = [&](int q, float c, float l, float4 acc) {
    const float inv = c == -INFINITY ? 0.0f : 1.0f / l;
    if (c == -INFINITY) acc = {0, 0, 0, 0};
    const int64_t r = out_row(a, s, hk, r0 + q);
    store4<E>(a.o + (r * D + d) * sizeof(E), acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (a.lse != nullptr && d == 0) a.lse[r] = c == -INFINITY ? -INFINITY : (c + log2f(l)) * kLn2;
  };
  auto fetch = [&](int i, int q, float& pc, float& pl, float4& z) {
    const float* part = cuts.parts + int64_t(i == 0 ? 2 * (b - 1) + 1 : 2 * (b + i - 1)) * part_size;
    pc = part[kRows * D + q];
    pl = part[kRows * (D + 1) + q];
    z = *reinterpret_cast<const float4*>(part + q * D + d);
  };
  auto merge = [](float& c, float& l, float4& acc, float pc, float pl, const float4& z) {
    // a piece without weights counts too, by a factor of 0: what it saw may not have been finite
    const float top = fmaxf(c, pc), base = top == -INFINITY ? 0.0f : top;
    const float f0 = __builtin_amdgcn_exp2f(c - base), f1 = __builtin_amdgcn_exp2f(pc - base);
    acc.x = acc.x * f0 + z.x * f1;
    acc.y = acc.y * f0 + z.y * f1;
    acc.z = acc.z * f0 + z.z * f1;
    acc.w = acc.w * f0 + z.w * f1;
    l = l * f0 + pl * f1;
    c = top;
  };
  const int step = share ? kSets : 1, side = share ? 1 : kSets;
  for (int q0 = y * side; q0 < rows; q0 += shares * side) {
    const int q = min(q0 + (share ? 0 : set), rows - 1);
    float4 acc = {0, 0, 0, 0};
    float l = 0.0f, c = -INFINITY;
    for (int i0 = share ? set : 0; i0 < pieces; i0 += kAhead * step) {
      float pc[kAhead], pl[kAhead];
      float4 z[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) fetch(min(i0 + k * step, pieces - 1), q, pc[k], pl[k], z[k]);
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k * step < pieces) merge(c, l, acc, pc[k], pl[k], z[k]);
    }
    if (!share) {
      if (q0 + set < rows) write(q, c, l, acc);
      continue;
    }
    acc_s[set][tid % kLanes] = acc;
    if (tid % kLanes == 0) l_s[set] = l, c_s[set] = c;
    __syncthreads();
    if (set == 0) {
      c = -INFINITY, l = 0.0f;
      acc = {0, 0, 0, 0};
#pragma unroll 1  // 94 registers instead of 130 at D = 64, so that more workgroups are there (drafts 67.5 -> 65 us)
      for (int v = 0; v < kSets; ++v) merge(c, l, acc, c_s[v], l_s[v], acc_s[v][tid]);
      write(q, c, l, acc);
    }
    __syncthreads();
  }
}

template <typename E, int D, int kWideRows, bool kByUnit = false>
__global__ __launch_bounds__(kJoinThreads, kByUnit ? 3 : 5) void join_kernel(AttnArgs a, int wide_share, int narrow_share) {
  // workgroups: `wide_share` for each cut of the wide kernel, then `narrow_share` for each of the narrow one (kByUnit: each unit)
  const int wide_blocks = a.wide.grid * wide_share;
  const bool wide = int(blockIdx.x) < wide_blocks;
  const Cuts& cuts = wide ? a.wide : a.narrow;
  const int at = wide ? blockIdx.x : blockIdx.x - wide_blocks, shares = wide ? wide_share : narrow_share;
  if (kByUnit && !wide) {
    // a unit that the narrow kernel has worked on has its entry
    for (int64_t i = at; i < int64_t(a.N) * a.Hkv * shares; i += gridDim.x - wide_blocks) {
      const int64_t unit = i / shares;
      const int n = int(unit / a.Hkv), hk = int(unit - int64_t(n) * a.Hkv);
      const int pieces = cuts.joins[2 * unit], b = cuts.joins[2 * unit + 1];   // asked for beside the lengths
      const int64_t rows = int64_t(seq_of(a, n).fresh) * a.group;
      if (rows == 0 || rows > kNarrowRows || pieces == 0) continue;
      const int y = int(i - unit * shares);
      if (pieces <= kManyPieces) {
        join_unit<E, D>(a, cuts, kNarrowRows, b, pieces, n, hk, 0, y, shares);
      } else {
        // 32 columns of a row at a time, so that more threads share its pieces
        for (int v = y; v < int(rows) * (D / 32); v += shares)
          join_unit<E, D, 32>(a, cuts, kNarrowRows, b, pieces, n, hk, 0, v / (D / 32), kNarrowRows, v % (D / 32) * 32);
      }
    }
    return;
  }
  const int b = at / shares, y = at - b * shares;
  const int pieces = cuts.joins[4 * b + 2];
  if (pieces == 0) return;
  const int n = cuts.joins[4 * b], hk = cuts.joins[4 * b + 1], r0 = cuts.joins[4 * b + 3];
  join_unit<E, D>(a, cuts, wide ? kWideRows : kNarrowRows, b, pieces, n, hk, r0, y, shares);
}

constexpr int kSlackPart = 32;  // a cut moves by up to this part of a stretch (an eighth of it to a 64th measured the same)

// Where the tiles of a cache in E come from: from memory straight into LDS, a wave's share of the rows (all in one page) per
// call. Another kind of cache brings its own: fetch asks for a tile, put, called once the tile before has been worked on, has
// it in LDS.
template <typename E, int D>
struct Direct {
  typedef AttnArgs Args;
  typedef E Cache;
  static constexpr int kMine = Wide<E, D>::kKeys / Wide<E, D>::kWaves;
  static constexpr int kTileBytes = Wide<E, D>::kTileBytes, kLoads = kTileBytes / 1024 / Wide<E, D>::kWaves;
  __device__ __forceinline__ void fetch(const AttnArgs& a, int32_t page, int hk, int32_t j, int row, uint32_t to, int lane) {
    const int64_t at = seg_offset<E, D>(a, page, hk, j);
    load_rows<E, D, false, kLoads>(a.kc + at, row, to + row * Tile<E, D>::kRowBytes, lane);
    load_rows<E, D, true, kLoads>(a.vc + at, row, to + kTileBytes + row * Tile<E, D>::kRowBytes, lane);
  }
  __device__ __forceinline__ void put(lds_u8*, int, int) {}
  __device__ __forceinline__ void arrived() { wait_loads<0>(); }
};

template <typename E, int D, typename S = Direct<E, D>>
__global__ __launch_bounds__((Wide<E, D, typename S::Cache>::kThreads),
                             (Wide<E, D, typename S::Cache>::kWaves / 4 * Wide<E, D, typename S::Cache>::kGroups)) void wide_kernel(
    typename S::Args a) {
  using C = typename S::Cache;
  using P = Wide<E, D, C>;
  __shared__ __align__(1024) unsigned char buf[4 * P::kTileBytes];
  __shared__ int odd_waves[P::kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // The row tiles, from memory or listed here.
  __shared__ int64_t own_sched[2 + kOwnTiles], own_starts[kFewSeqs], scan_part[P::kWaves];
  __shared__ RowTile own_tiles[kOwnTiles];
  if (a.own_list) {
    list_row_tiles<P, P::kThreads>(a, scan_part, own_sched, own_tiles, own_starts);
    __syncthreads();
  }
  const int64_t* const sched = a.own_list ? own_sched : a.sched;
  const int64_t count = uniform(sched[0]), per_head = uniform(sched[1]);
  const int64_t total = per_head * a.Hkv;
  // Workgroups go to the 8 XCDs in turn: neighbouring stretches, which read the same keys, share an L2.
  const int grid = P::kGroups > 1 && total < int64_t(P::kShort) * a.wide.grid ? min(a.wide.grid, kCus) : a.wide.grid;
  const int b = int(blockIdx.x) < grid ? int(blockIdx.x % 8) * (grid / 8) + int(blockIdx.x / 8) : int(blockIdx.x);
  if (tid == 0) a.wide.joins[4 * b + 2] = 0;
  if (total == 0) return;
  // Short stretches, so that small calls spread: one sequence of 500 keys and 500 rows at D = 256 takes 30 us with 5 tiles
  // at least, 27 with 3, 28 with 1.
  const Line line(total, grid, 1 + P::kOver / 4);
  const int64_t* const before = sched + 2;
  // The unit that holds position `at`: key head, row tile, start.
  auto find = [&](int64_t at, int& head, int& tile, int64_t& start, int64_t& size) {
    head = __builtin_amdgcn_readfirstlane(int(at / per_head));
    const int64_t in = at - head * per_head;
    // the last row tile that starts at or before `in`, 64 probes at a time
    int64_t lo = 0, len = count;
    while (len > 1) {
      const int64_t step = (len + 63) / 64, probe = lo + lane * step;
      const int hits = __popcll(__ballot(probe < lo + len && before[min(probe, count - 1)] <= in));
      const int64_t next = lo + max(hits - 1, 0) * step;
      len = min(step, lo + len - next);
      lo = next;
    }
    tile = __builtin_amdgcn_readfirstlane(int(lo));
    const int64_t at_tile = uniform(before[tile]);
    start = at_tile + head * per_head;
    size = (tile + 1 < count ? uniform(before[tile + 1]) : per_head) - at_tile;
  };
  // A cut costs a write and a read of a whole output tile, so one that falls near an end of a unit moves there (and one
  // in its fixed part always moves to the start).
  const int64_t slack = total / line.parts / kSlackPart, head = max(slack, int64_t(P::kOver));
  auto snap = [&](int64_t at, int64_t start, int64_t size) {
    return at - start <= head ? start : start + size - at <= slack ? start + size : at;
  };
  int hk, rt, other_hk, other_rt;
  int64_t start, length, pos = line.start(b), end = line.start(b + 1);
  if (pos >= total) return;
  if (end < total) {
    find(end, other_hk, other_rt, start, length);
    end = snap(end, start, length);
  }
  find(pos, hk, rt, start, length);
  pos = snap(pos, start, length);
  if (pos >= end) return;
  if (pos == start + length) {
    start = pos;
    if (++rt >= count) rt = 0, ++hk;
  }
  Wave<E, D, D, C> w;
  S src;
  lds_u8* const tiles_at = (lds_u8*)buf;
  const uint32_t buf_at = uint32_t(uintptr_t(tiles_at));
  const_row_tile* const list = (const_row_tile*)a.row_tiles;

  // A unit: a row tile of a key head, and the part of its tiles of keys that is this stretch's.
  struct Unit {
    Seq s;
    Span x;
    int32_t n, hk, rows, r0, in, out, t0, t1;  // in, out: where the stretch enters the unit and leaves it
  };
  auto describe = [&](const RowTile& d, int head, int64_t from, int64_t left) {
    Unit u;
    u.n = d.n;
    u.hk = head;
    u.s = {d.start, d.fresh, d.kv};
    u.rows = d.fresh * a.group;
    u.r0 = d.r0;
    u.x.first = max(d.kv - d.fresh + d.r0 / a.group, -1);
    u.x.last = max(d.kv - d.fresh + (min(d.r0 + P::kRows, u.rows) - 1) / a.group, -1);
    u.x.lo = d.lo;
    u.x.hi = d.hi;
    u.in = int32_t(from);
    u.out = int32_t(min(int64_t(d.hi - d.lo + P::kOver), from + left));
    u.t0 = max(u.in - P::kOver, 0);
    u.t1 = max(u.out - P::kOver, 0);
    return u;
  };
  auto tile_of = [&](int at) {
    RowTile d;
    if (a.own_list) {
      const RowTile& o = own_tiles[at];
      d.n = __builtin_amdgcn_readfirstlane(o.n);
      d.r0 = __builtin_amdgcn_readfirstlane(o.r0);
      d.start = __builtin_amdgcn_readfirstlane(o.start);
      d.fresh = __builtin_amdgcn_readfirstlane(o.fresh);
      d.kv = __builtin_amdgcn_readfirstlane(o.kv);
      d.lo = __builtin_amdgcn_readfirstlane(o.lo);
      d.hi = __builtin_amdgcn_readfirstlane(o.hi);
    } else {
      d = *(const RowTile*)(list + at);
    }
    return d;
  };

  // this wave's share of a tile of keys: rows mine_at .., all in one page, looked up one tile ahead
  constexpr int kMine = P::kKeys / P::kWaves;
  static_assert(kMine <= kSeg && kSeg % kMine == 0, "one page");
  const int mine_at = wave * kMine;
  int32_t page;
  auto look_up = [&](const Unit& u, int32_t t) {
    page = seg_page(a, (const_i32*)(a.table + int64_t(u.n) * a.width), max((u.s.kv - 1) >> a.lps, 0),
                    (u.x.lo + t) * P::kKeys + mine_at);
  };
  auto load = [&](const Unit& u, int32_t t, uint32_t to) {
    src.fetch(a, page, u.hk, (u.x.lo + t) * P::kKeys + mine_at, mine_at, to, lane);
  };

  uint32_t half = 0;
  bool there = false;   // the unit's first tile has been asked for
  int64_t from = pos - start;
  for (;;) {
    const Unit u = describe(tile_of(rt), hk, from, end - pos);
    if (!there) {
      look_up(u, u.t0);
      load(u, u.t0, buf_at + half);
      src.put(tiles_at + half, mine_at, lane);
    }
    look_up(u, u.t0 + 1);
    const int32_t w0 = u.r0 + wave * 32;   // this wave's rows
    w.queries(a, u.s, u.hk, w0 + (lane & 31), u.rows, lane);
    w.start(a, u.s, w0 + (lane & 31), u.rows);
    const int64_t after = pos + (u.out - u.in);
    const bool more = after < end;
    const bool busy = w0 < u.rows;
    const int32_t first = max(u.s.kv - u.s.fresh + min(w0, u.rows - 1) / a.group, -1);   // the positions of this wave's rows
    const int32_t last = max(u.s.kv - u.s.fresh + min(w0 + 31, u.rows - 1) / a.group, -1);
    for (int32_t t = u.t0; t < u.t1; ++t) {
      src.arrived();
      __syncthreads();   // the tile is there, and every wave is done with the other buffer
      const uint32_t other = buf_at + (half ^ 2 * P::kTileBytes);
      if (t + 1 < u.t1) {
        load(u, t + 1, other);
        look_up(u, t + 2);
      } else if (more) {
        // the next unit's first tile arrives while this unit ends
        const bool turn = rt + 1 >= count;
        const Unit v = describe(tile_of(turn ? 0 : rt + 1), turn ? hk + 1 : hk, 0, end - after);
        look_up(v, v.t0);
        load(v, v.t0, other);
      }
      const int32_t kv0 = (u.x.lo + t) * P::kKeys;
      const bool none = !busy || kv0 > last || (a.window > 0 && kv0 + P::kKeys - 1 <= first - a.window);
      const bool full = kv0 + P::kKeys - 1 <= first && (a.window == 0 || kv0 > last - a.window);
      if (kv0 + P::kKeys - 1 > u.x.first || (a.window > 0 && kv0 <= u.x.last - a.window)) {
        // some row of the workgroup does not see all of it
        lds_u8* const vt = tiles_at + half + P::kTileBytes;
        const bool odd = __any(any_odd<C, P::kTileBytes, P::kThreads>(vt, tid));
        if (lane == 0) odd_waves[wave] = odd;
        __syncthreads();
        int found = 0;
        for (int y = 0; y < P::kWaves; ++y) found |= odd_waves[y];
        if (found) {
          if (!none) w.template mark<P::kKeys>(vt, kv0, lane, 0);
          __syncthreads();
          clean<C, P::kTileBytes, P::kThreads>(vt, tid);
          __syncthreads();
        }
      }
      if (!none) {
        typename Operand<E, C>::type p[P::kKeys / 16];
        w.template scores<P::kKeys>(a, tiles_at + half, kv0, full, lane, p, Nothing{});
        w.template values<P::kKeys>(tiles_at + half + P::kTileBytes, p, lane);
      }
      if (t + 1 < u.t1 || more) src.put(tiles_at + (half ^ 2 * P::kTileBytes), mine_at, lane);
      half ^= 2 * P::kTileBytes;
    }

    const float l_all = w.finish();
    const bool whole = u.t0 == 0 && u.t1 == u.x.hi - u.x.lo;
    const int32_t r = w0 + (lane & 31), h = lane >> 5;
    if (whole) {
      if (r < u.rows) {
        const float inv = w.c == -INFINITY ? 0.0f : 1.0f / l_all;
        const int64_t at = out_row(a, u.s, u.hk, r);
        store_row<E, D>(a.o + at * D * sizeof(E), w.o, inv, h);
        if (a.lse != nullptr && h == 0) a.lse[at] = w.c == -INFINITY ? -INFINITY : (w.c + log2f(l_all)) * kLn2;
      }
    } else {
      float* const part = a.wide.parts + int64_t(2 * b + (u.t0 == 0 ? 1 : 0)) * part_floats<D>(P::kRows);
      const int q = wave * 32 + (lane & 31);
      if (r < u.rows) {
        store_row<float, D>(reinterpret_cast<uint8_t*>(part + q * D), w.o, 1.0f, h);
        if (h == 0) {
          part[P::kRows * D + q] = w.c;
          part[P::kRows * (D + 1) + q] = l_all;
        }
      }
      // the first cut of this unit: the one before is not within it (or has moved to its start)
      if (tid == 0 && u.t0 > 0 && line.start(b - 1) <= pos - u.in + head) {
        const int64_t ends = pos - u.in + (u.x.hi - u.x.lo + P::kOver);
        a.wide.joins[4 * b] = u.n;
        a.wide.joins[4 * b + 1] = u.hk;
        a.wide.joins[4 * b + 3] = u.r0;
        a.wide.joins[4 * b + 2] = int32_t(1 + line.before(ends - slack) - b);
      }
    }
    if (!more) break;
    pos = after;
    from = 0;
    there = true;
    if (++rt >= count) rt = 0, ++hk;
  }
}

// |scale| log2 e, which multiplies the scores.
float log2_scale(float scale) { return std::fabs(scale) * kLog2e; }

rglru_status_t check(const rglru_paged_shape_t& s) {
  if (!valid_pages(s) || !valid_table(s) || !valid_io(s) || s.kv_heads < 1 || s.q_heads < s.kv_heads ||
      s.q_heads > (1 << 14) || s.q_heads % s.kv_heads != 0 || s.n_tokens * s.q_heads > (int64_t(1) << 31) - (1 << 16) ||
      s.head_dim < 1 || s.head_dim > (1 << 16) || s.window < 0 || !std::isfinite(log2_scale(s.scale)) ||
      row_stride(s.q_stride, int64_t(s.q_heads) * s.head_dim) < 0)
    return RGLRU_ERR_INVALID_ARGUMENT;
  if (s.head_dim != 64 && s.head_dim != 128 && s.head_dim != 256) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

// The largest number of tokens and of rows of one sequence that the caller allows.
int64_t most_tokens(const rglru_paged_shape_t& s) { return s.max_new > 0 && s.max_new < s.n_tokens ? s.max_new : s.n_tokens; }
int64_t most_rows(const rglru_paged_shape_t& s) { return most_tokens(s) * (s.q_heads / s.kv_heads); }

// The largest number of sequences of few rows in a batch of n_tokens where the others have most_tokens at most, and those
// have more than kNarrowRows rows.
int64_t most_few(const rglru_paged_shape_t& s) {
  const int64_t longest = most_tokens(s), few = kNarrowRows / (s.q_heads / s.kv_heads);
  const int64_t x = (s.n_seqs * longest - s.n_tokens) / (longest - few);
  return x < 0 ? 0 : x < s.n_seqs ? x : s.n_seqs;
}

// A call whose sequences may all have at most kNarrowRows rows runs the narrow
// kernel alone; any other one the wide kernel, and before it the narrow kernel for the
// sequences of few rows unless those are few themselves (kFewSeqs sequences, few_units
// pairs of a sequence of few rows and a key head). The workspace has room for the narrow kernel wherever a
// call of fewer tokens would run it, so one of the largest size serves all.
struct Plan {
  bool narrow, wide, own_list;
  int narrow_grid, wide_grid;  // stretches: workgroups (of the wide kernel a multiple of 8) or their waves
  int64_t max_tiles;           // row tiles of the wide kernel at most
  size_t narrow_joins, narrow_parts, wide_joins, wide_parts, row_tiles, sched, bytes;  // offsets and size of the workspace
};

// N: the narrow kernel's traits, its tiles of `keys`; W: the wide kernel's.
template <typename N, typename W, int D>
Plan plan_of(const rglru_paged_shape_t& s, int narrow_keys, int few_units) {
  Plan p = {};
  p.wide = most_rows(s) > kNarrowRows;
  const bool room = !p.wide || s.n_seqs > kFewSeqs || int64_t(s.n_seqs) * s.kv_heads > few_units;
  p.narrow = !p.wide || s.n_seqs > kFewSeqs || most_few(s) * s.kv_heads > few_units;
  const int64_t group = s.q_heads / s.kv_heads;
  const int64_t keys = int64_t(s.max_pages) * s.page_size;
  const int64_t seqs = s.n_seqs < s.n_tokens ? s.n_seqs : s.n_tokens;
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t start = at;
    at += round_up(bytes, 256);
    return start;
  };
  // no more workgroups than there can be tiles
  auto grid_of = [](int64_t most, int64_t units, int64_t tiles) {
    return int(units >= most || tiles >= most || units * tiles >= most ? most : units * tiles > 0 ? units * tiles : 1);
  };
  if (room) {
    p.narrow_grid = grid_of(256 * N::kGroups, seqs * s.kv_heads, ceil_div(ceil_div(keys, narrow_keys), N::kWaves)) * N::kStretches;
    const size_t units = size_t(s.n_seqs) * s.kv_heads;
    p.narrow_joins = take(N::kStretches > 1 ? units * 8 : size_t(p.narrow_grid) * 16);
    p.narrow_parts = take(size_t(p.narrow_grid) * 2 * part_floats<D>(kNarrowRows) * 4);
  }
  if (p.wide) {
    p.max_tiles = ceil_div(s.n_tokens * group, W::kRows) + seqs;
    p.own_list = !p.narrow && p.max_tiles <= kOwnTiles;
    p.wide_grid = (grid_of(256 * W::kGroups, p.max_tiles * s.kv_heads, ceil_div(keys, W::kKeys)) + 7) / 8 * 8;
    p.row_tiles = take(size_t(p.max_tiles) * sizeof(RowTile));
    p.sched = take(size_t(2 + p.max_tiles + s.n_seqs) * 8);
    p.wide_joins = take(size_t(p.wide_grid) * 16);
    p.wide_parts = take(size_t(p.wide_grid) * 2 * part_floats<D>(W::kRows) * 4);
  }
  if (!p.narrow) p.narrow_grid = 0;
  p.bytes = at;
  return p;
}

// Where a call's pieces lie in its workspace.
void lay_out(AttnArgs& a, const Plan& p, uint8_t* workspace) {
  a.narrow = {reinterpret_cast<int32_t*>(workspace + p.narrow_joins), reinterpret_cast<float*>(workspace + p.narrow_parts),
              p.narrow_grid};
  a.wide = {reinterpret_cast<int32_t*>(workspace + p.wide_joins), reinterpret_cast<float*>(workspace + p.wide_parts),
            p.wide_grid};
  a.sched = reinterpret_cast<int64_t*>(workspace + p.sched);
  a.row_tiles = reinterpret_cast<RowTile*>(workspace + p.row_tiles);
  a.max_tiles = int32_t(p.max_tiles);
  a.own_list = p.own_list;
  a.least_rows = p.narrow ? kNarrowRows : 0;
}

template <typename E, int D, typename W, bool kByUnit = false>
void join(const rglru_paged_shape_t& s, const AttnArgs& a, const Plan& p, hipStream_t st) {
  // A pass over kPass rows costs the latency of its reads, 2 to 3 us: one pass (rows of few pieces; with many, a row a pass).
  constexpr int kPass = kJoinThreads * 4 / D;
  const int wide_share = W::kRows / kPass;
  int narrow_share = int(p.wide ? ceil_div(kNarrowRows, kPass) : most_rows(s));
  int64_t narrow = !kByUnit ? p.narrow_grid : p.narrow ? int64_t(s.n_seqs) * s.kv_heads : 0;
  if (kByUnit && !p.wide && narrow > 0) {
    // few units have many pieces each: more workgroups for a unit's rows
    const int64_t pass = ceil_div(most_rows(s), kPass), spread = ceil_div(4 * kCus, narrow), most = most_rows(s) * (D / 32);
    narrow_share = int(spread < pass ? pass : spread < most ? spread : most);
  }
  narrow *= narrow_share;
  if (kByUnit && narrow > (1 << 20)) narrow = 1 << 20;   // they take further units in turn
  join_kernel<E, D, W::kRows, kByUnit><<<unsigned(p.wide_grid * wide_share + narrow), kJoinThreads, 0, st>>>(a, wide_share,
                                                                                                       narrow_share);
}

void set_args(AttnArgs& a, const rglru_paged_shape_t& s, const int32_t* cu_seqlens, const int32_t* kv_lens,
              const int32_t* block_table, const void* q, const void* k_cache, const void* v_cache, void* o, float* lse) {
  a.cu = cu_seqlens;
  a.kv_lens = kv_lens;
  a.table = block_table;
  a.q = static_cast<const uint8_t*>(q);
  a.kc = static_cast<const uint8_t*>(k_cache);
  a.vc = static_cast<const uint8_t*>(v_cache);
  a.o = static_cast<uint8_t*>(o);
  a.lse = lse;
  a.T = int32_t(s.n_tokens);
  a.q_stride = row_stride(s.q_stride, int64_t(s.q_heads) * s.head_dim);
  a.n_pages = int32_t(s.n_pages);
  a.N = s.n_seqs;
  a.width = s.max_pages;
  a.lps = log2_of(s.page_size);
  a.Hq = s.q_heads;
  a.Hkv = s.kv_heads;
  a.group = s.q_heads / s.kv_heads;
  a.window = s.window < int64_t(s.max_pages) * s.page_size ? s.window : 0;  // a window as long as the row hides nothing
  a.scale2 = s.scale == 0.0f ? 1.0f : log2_scale(s.scale);
  a.q_sign = s.scale > 0.0f ? 1 : s.scale < 0.0f ? -1 : 0;
}

// Calls f<E, D>(...) for the shape's type and head width.
#define RGLRU_PAGED_DISPATCH(s, f, ...)                                                                  \
  ((s).io_dtype == RGLRU_IO_BF16                                                                         \
       ? ((s).head_dim == 64 ? f<uint16_t, 64>(__VA_ARGS__)                                              \
                             : (s).head_dim == 128 ? f<uint16_t, 128>(__VA_ARGS__) : f<uint16_t, 256>(__VA_ARGS__)) \
       : ((s).head_dim == 64 ? f<float, 64>(__VA_ARGS__)                                                 \
                             : (s).head_dim == 128 ? f<float, 128>(__VA_ARGS__) : f<float, 256>(__VA_ARGS__)))

}  // namespace
}  // namespace paged
}  // namespace rglru
