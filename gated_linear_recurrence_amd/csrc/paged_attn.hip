// Attention of new tokens over a paged key/value cache (include/paged_attn.h).
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
  int32_t* joins;  // [grid][4]: sequence, key head, pieces (0: none) and first row of what the cut before workgroup b parted
  float* parts;    // [grid][2]: partial results of a workgroup's first and last unit
  int32_t grid;
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
template <typename E, int D, int kSlice = D>
struct Wave {
  using L = Tile<E, kSlice>;
  static constexpr int kSlices = D / kSlice;
  static constexpr int kHeld = kSlices > 1 ? D / 32 : D / 16;  // operands of queries in registers; the others in LDS, at `rest`
  static constexpr int kRestBytes = (D / 16 - kHeld) * 64 * int(sizeof(Frag<E>));
  lds_u8* rest;
  Frag<E> q[D / 16];
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
      q[x].w = 0;
      if (live) {
        // in pieces of 16 bytes, which is what the rows are aligned to
        const u32x4* const from = reinterpret_cast<const u32x4*>(src + (x * 16 + h * 8) * sizeof(E));
        if constexpr (sizeof(E) == 2) q[x].w = from[0];
        else q[x].w = __builtin_shufflevector(from[0], from[1], 0, 1, 2, 3, 4, 5, 6, 7);
      }
    }
  }

  __device__ __forceinline__ void start(const AttnArgs& a, const Seq& s, int32_t r, int32_t rows) {
    if (a.q_sign <= 0) {
      const uint32_t keep = a.q_sign == 0 ? 0u : ~0u, flip = a.q_sign < 0 ? Frag<E>::kSigns : 0u;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) q[x].w = (q[x].w & keep) ^ flip;
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
    auto* const to = (__attribute__((address_space(3))) u32x4*)(rest + i * 64 * int(sizeof(Frag<E>)));
#pragma unroll
    for (int j = 0; j < int(sizeof(Frag<E>)) / 16; ++j)
      to[j * 64 + lane] = reinterpret_cast<const u32x4*>(&q[kHeld + i])[j];
  }
  __device__ __forceinline__ Frag<E> get_query(int i, int lane) const {
    Frag<E> f;
    const auto* const from = (const __attribute__((address_space(3))) u32x4*)(rest + i * 64 * int(sizeof(Frag<E>)));
#pragma unroll
    for (int j = 0; j < int(sizeof(Frag<E>)) / 16; ++j) reinterpret_cast<u32x4*>(&f)[j] = from[j * 64 + lane];
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
                                         Frag<E>* p, Done done, Ready ready = {}) {
    const int h = lane >> 5;
    f32x16 s[BN / 32];
    {
      // product i: keys of subtile i / (D / 16), elements 16 (i % (D / 16)) on; operands are read kAhead products early
      constexpr int kSteps = D / 16, kAll = BN / 32 * kSteps, kAhead = sizeof(E) == 2 ? 4 : 2;
      constexpr int kOne = kSteps / kSlices;
      static_assert(kSlices == 1 || (BN == 32 && kAhead < kOne), "a slice's products follow each other");
      const int r = lane & 31;
      int at = r * L::kRowBytes + (sizeof(E) == 2 ? (h ^ L::swz_k(r)) * 16 : ((2 * h) ^ L::swz_k(r)) * 16);
      fresh_value(at);
      Frag<E> k[kAhead], z[kAhead];
      auto fetch = [&](int i) {
        const int b = i / kSteps, x = i % kOne;
        const lds_u8* p = kt + (b + i % kSteps / kOne) * 32 * L::kRowBytes;
        if (kSlices > 1 && x == 0) ready(i / kOne);
        if (i % kSteps >= kHeld) z[i % kAhead] = get_query(i % kSteps - kHeld, lane);
        if constexpr (sizeof(E) == 2) {
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
        p[2 * b + y] = pack(w, E{});
      }
    l += sum;
  }

  // Adds BN weighted values to the output; ready(c) and done(c) as above, of several slices.
  template <int BN, typename Ready = Nothing, typename Done = Nothing>
  __device__ __forceinline__ void values(const lds_u8* vt, const Frag<E>* p, int lane, Ready ready = {}, Done done = {}) {
    constexpr int kSteps = BN / 16, kAll = D / 32 * kSteps, kAhead = sizeof(E) == 2 ? 4 : 2, kOne = kAll / kSlices;
    static_assert(kSlices == 1 || kAhead < kOne, "a slice's products follow each other");
    int start = value_at(lane);
    fresh_value(start);
    Frag<E> v[kAhead];
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
    if constexpr (sizeof(E) == 2) {
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
  __device__ __forceinline__ Frag<E> value_frag(const lds_u8* vt, int x, int y, int start) const {
    Frag<E> v;
    constexpr int kCols = kSlice / 32;
    const int at = (start ^ (x % kCols * 32 * int(sizeof(E)))) + (x / kCols * BN + y * 16) * L::kRowBytes;
    if constexpr (sizeof(E) == 2) {
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
    Frag<E> see[BN / 16];
#pragma unroll
    for (int y = 0; y < BN / 16; ++y) {
      float one[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int32_t j = kv0 + 16 * y + 8 * (r / 4) + r % 4 + 4 * (lane >> 5);
        one[r] = j >= lo && j <= hi ? 1.0f : 0.0f;
      }
      see[y] = pack(one, E{});
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
constexpr int kNarrowRows = 32, kNarrowKeys = 32, kNarrowOver = 6;

// In a call that needs the wide kernel it takes the sequences of few rows too where there are at most kFewSeqs sequences and
// kFewUnits (sequence of few rows, key head) pairs: it saves a launch, but works through such a unit as slowly as through
// one of many rows. 618 calls of a chunk of 200 or 1000 tokens and 1 to 15 single tokens, all after 200 to 8000 tokens, 1
// to 16 key heads, timed with the wide kernel alone and with both: taking the better of the two by this rule costs 1.6 %
// more than by the clock in bf16 at D = 64 and 2.2 to 2.8 % in float32 (without the second bound 5 and 7 to 13 %), 0.2 %
// in bf16 at D = 128 and 256, whose best bound is past what was measured (240). A chunk of 1000 after 2000 at D = 128, 4
// key heads, alone and both: beside 15 single tokens 56 and 60 us, in float32 273 and 239; beside 47 87 and 78.
constexpr int kFewSeqs = 16;
template <typename E, int D>
constexpr int kFewUnits = sizeof(E) == 4 ? 24 : D == 64 ? 64 : 256;

template <typename E, int D>
struct Narrow {
  static constexpr int kTileBytes = kNarrowKeys * D * int(sizeof(E));
  // 128 KB of LDS per CU, four waves in a workgroup. Up to 8 KB a tile each wave has two buffers of keys and two of
  // values (and there are two workgroups at 4 KB), at 16 KB one of each, at 32 KB one for both. kGroups also tells
  // the compiler how many waves share a SIMD: with two it keeps the output out of the accumulation registers, which it
  // copies to and fro otherwise (D = 64: 22.4 -> 21 us for 16 sequences of 2000 keys).
  static constexpr int kWaves = 4;
  static constexpr int kBuffers = kTileBytes <= 8192 ? 4 : 32768 / kTileBytes;
  static constexpr int kGroups = kTileBytes == 4096 ? 2 : 1;
  static constexpr int kThreads = kWaves * 64;
  // The one buffer holds four slices of columns, each loaded anew as soon as it is read: those of the values take the
  // place of those of the keys and the other way round. Half of the queries lie in LDS, as the registers would not hold
  // them and the output (float32, D = 256, 64 sequences of 8000 keys, 2 key heads: whole tiles in turn 3.9 TB/s, slices
  // 4.4, with half of the queries in LDS 5.1, now that no register spills 5.7).
  static constexpr int kSlice = kBuffers == 1 ? D / 4 : D;
};

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

// Length of a unit of a sequence in the line.
__device__ __forceinline__ int32_t narrow_size(const AttnArgs& a, const Seq& s) {
  if (s.fresh == 0 || int64_t(s.fresh) * a.group > kNarrowRows) return 0;
  const Span x = span_of<kNarrowKeys>(a, s, 0, s.fresh * a.group - 1);
  return x.hi - x.lo + kNarrowOver;
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
template <typename E, int D>
struct Wide {
  static constexpr bool kBf16 = sizeof(E) == 2;
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
  static constexpr int kOver = !kBf16 ? 1 : D == 256 ? 9 : D == 128 ? 4 : 5;
  static constexpr int kTileBytes = kKeys * D * int(sizeof(E));
  static constexpr int kLoads = kTileBytes / 1024 / kWaves;  // per wave, keys and values each
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
constexpr int kOwnTiles = 256;
constexpr int kCus = 256;   // of the card

template <typename W>
__global__ __launch_bounds__(kSchedThreads) void sched_kernel(AttnArgs a) {
  __shared__ int64_t part[kSchedThreads / 64];
  list_row_tiles<W, kSchedThreads>(a, part, a.sched, a.row_tiles, a.sched + 2 + a.max_tiles);
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

// Merges the pieces of every unit that was cut, in the order of the keys. A
// row takes D / 4 threads; the other threads of a workgroup take further rows
// or, where there are many pieces, further pieces of the same row.
constexpr int kJoinThreads = 256;

template <typename E, int D, int kWideRows>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(AttnArgs a, int wide_share, int narrow_share) {
  constexpr int kLanes = D / 4, kSets = kJoinThreads / kLanes, kAhead = 8, kShare = 16;
  __shared__ float4 acc_s[kSets][kLanes];
  __shared__ float l_s[kSets], c_s[kSets];
  // workgroups: `wide_share` for each cut of the wide kernel, then `narrow_share` for each of the narrow one
  const int wide_blocks = a.wide.grid * wide_share;
  const bool wide = int(blockIdx.x) < wide_blocks;
  const Cuts& cuts = wide ? a.wide : a.narrow;
  const int at = wide ? blockIdx.x : blockIdx.x - wide_blocks, shares = wide ? wide_share : narrow_share;
  const int b = at / shares, y = at - b * shares, tid = threadIdx.x;
  const int pieces = cuts.joins[4 * b + 2];
  if (pieces == 0) return;
  const int n = cuts.joins[4 * b], hk = cuts.joins[4 * b + 1], r0 = cuts.joins[4 * b + 3];
  const Seq s = seq_of(a, n);
  const int kRows = wide ? kWideRows : kNarrowRows;
  const int64_t part_size = int64_t(kRows) * (D + 2);
  const int rows = min(kRows, s.fresh * a.group - r0);
  // The sets share a row's pieces where there are many and that takes fewer reads in a row than a set per row.
  const bool share = pieces > kShare && (rows + shares - 1) / shares * kAhead < pieces;
  const int set = tid / kLanes, d = (tid % kLanes) * 4;
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
    if (d == 0) l_s[set] = l, c_s[set] = c;
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

constexpr int kSlackPart = 32;  // a cut moves by up to this part of a stretch (an eighth of it to a 64th measured the same)

template <typename E, int D>
__global__ __launch_bounds__((Wide<E, D>::kThreads), (Wide<E, D>::kWaves / 4 * Wide<E, D>::kGroups)) void wide_kernel(AttnArgs a) {
  using P = Wide<E, D>;
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
  Wave<E, D> w;
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
    const int64_t at = seg_offset<E, D>(a, page, u.hk, (u.x.lo + t) * P::kKeys + mine_at);
    load_rows<E, D, false, P::kLoads>(a.kc + at, mine_at, to + mine_at * Tile<E, D>::kRowBytes, lane);
    load_rows<E, D, true, P::kLoads>(a.vc + at, mine_at, to + P::kTileBytes + mine_at * Tile<E, D>::kRowBytes, lane);
  };

  uint32_t half = 0;
  bool there = false;   // the unit's first tile has been asked for
  int64_t from = pos - start;
  for (;;) {
    const Unit u = describe(tile_of(rt), hk, from, end - pos);
    if (!there) {
      look_up(u, u.t0);
      load(u, u.t0, buf_at + half);
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
      wait_loads<0>();
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
        const bool odd = __any(any_odd<E, P::kTileBytes, P::kThreads>(vt, tid));
        if (lane == 0) odd_waves[wave] = odd;
        __syncthreads();
        int found = 0;
        for (int y = 0; y < P::kWaves; ++y) found |= odd_waves[y];
        if (found) {
          if (!none) w.template mark<P::kKeys>(vt, kv0, lane, 0);
          __syncthreads();
          clean<E, P::kTileBytes, P::kThreads>(vt, tid);
          __syncthreads();
        }
      }
      if (!none) {
        Frag<E> p[P::kKeys / 16];
        w.template scores<P::kKeys>(a, tiles_at + half, kv0, full, lane, p, Nothing{});
        w.template values<P::kKeys>(tiles_at + half + P::kTileBytes, p, lane);
      }
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
// kernel alone (32 sequences of 4096 keys, 32 rows on each of 4 key heads of
// 128: 60 us, the wide kernel 65); any other one the wide kernel, and before it
// the narrow kernel for the sequences of few rows unless those are few themselves
// (kFewSeqs, kFewUnits). The workspace has room for the narrow kernel wherever a
// call of fewer tokens would run it, so one of the largest size serves all.
struct Plan {
  bool narrow, wide, own_list;
  int narrow_grid, wide_grid;  // workgroups; of the wide kernel a multiple of 8
  int64_t max_tiles;           // row tiles of the wide kernel at most
  size_t narrow_joins, narrow_parts, wide_joins, wide_parts, row_tiles, sched, bytes;  // offsets and size of the workspace
};

template <typename E, int D>
Plan plan_of(const rglru_paged_shape_t& s) {
  using W = Wide<E, D>;
  Plan p = {};
  p.wide = most_rows(s) > kNarrowRows;
  const bool room = !p.wide || s.n_seqs > kFewSeqs || int64_t(s.n_seqs) * s.kv_heads > kFewUnits<E, D>;
  p.narrow = !p.wide || s.n_seqs > kFewSeqs || most_few(s) * s.kv_heads > kFewUnits<E, D>;
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
    using P = Narrow<E, D>;
    p.narrow_grid = grid_of(256 * P::kGroups, seqs * s.kv_heads, ceil_div(ceil_div(keys, kNarrowKeys), P::kWaves));
    p.narrow_joins = take(size_t(p.narrow_grid) * 16);
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

template <typename E, int D>
size_t bytes_of(const rglru_paged_shape_t& s) {
  return plan_of<E, D>(s).bytes;
}

template <typename E, int D>
void launch(const rglru_paged_shape_t& s, AttnArgs a, uint8_t* workspace, hipStream_t st) {
  using W = Wide<E, D>;
  const Plan p = plan_of<E, D>(s);
  a.narrow = {reinterpret_cast<int32_t*>(workspace + p.narrow_joins), reinterpret_cast<float*>(workspace + p.narrow_parts),
              p.narrow_grid};
  a.wide = {reinterpret_cast<int32_t*>(workspace + p.wide_joins), reinterpret_cast<float*>(workspace + p.wide_parts),
            p.wide_grid};
  a.sched = reinterpret_cast<int64_t*>(workspace + p.sched);
  a.row_tiles = reinterpret_cast<RowTile*>(workspace + p.row_tiles);
  a.max_tiles = int32_t(p.max_tiles);
  a.own_list = p.own_list;
  a.least_rows = p.narrow ? kNarrowRows : 0;
  if (p.narrow) narrow_kernel<E, D><<<unsigned(p.narrow_grid + p.wide), Narrow<E, D>::kThreads, 0, st>>>(a);
  if (p.wide) {
    if (!p.narrow && !p.own_list) sched_kernel<W><<<1, kSchedThreads, 0, st>>>(a);
    wide_kernel<E, D><<<unsigned(p.wide_grid), W::kThreads, 0, st>>>(a);
  }
  // A pass over kPass rows costs the latency of its reads, 2 to 3 us: one pass (rows of few pieces; with many, a row a pass).
  constexpr int kPass = kJoinThreads * 4 / D;
  const int wide_share = W::kRows / kPass, narrow_share = int(p.wide ? ceil_div(kNarrowRows, kPass) : most_rows(s));
  join_kernel<E, D, W::kRows><<<unsigned(p.wide_grid * wide_share + p.narrow_grid * narrow_share), kJoinThreads, 0, st>>>(
      a, wide_share, narrow_share);
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
  a.cu = cu_seqlens;
  a.kv_lens = kv_lens;
  a.table = block_table;
  a.q = static_cast<const uint8_t*>(q);
  a.kc = static_cast<const uint8_t*>(k_cache);
  a.vc = static_cast<const uint8_t*>(v_cache);
  a.o = static_cast<uint8_t*>(o);
  a.lse = lse;
  a.T = int32_t(s.n_tokens);
  a.q_stride = stride;
  a.n_pages = int32_t(s.n_pages);
  a.N = s.n_seqs;
  a.width = s.max_pages;
  a.lps = paged::log2_of(s.page_size);
  a.Hq = s.q_heads;
  a.Hkv = s.kv_heads;
  a.group = s.q_heads / s.kv_heads;
  a.window = s.window < int64_t(s.max_pages) * s.page_size ? s.window : 0;  // a window as long as the row hides nothing
  a.scale2 = s.scale == 0.0f ? 1.0f : paged::log2_scale(s.scale);
  a.q_sign = s.scale > 0.0f ? 1 : s.scale < 0.0f ? -1 : 0;
  RGLRU_PAGED_DISPATCH(s, paged::launch, s, a, static_cast<uint8_t*>(workspace), static_cast<hipStream_t>(stream));
  return launch_status();
}
