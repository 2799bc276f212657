// Attention of new tokens over a 4-bit paged cache (include/paged_q4.h).
//
// The formula and the treatment of rows, masks and pieces are those of
// paged_attn_core.h; a cache of 4.25 bits an element changes where the time goes.
//
// Many rows (chunks of a prompt): bound by the matrix cores as over a bf16 cache.
// The wide kernel runs as it is on tiles of bf16 in LDS; only their source
// differs: each wave fetches its share of the codes into registers while the tile
// before is worked on, and writes the values, which bf16 holds exactly, once for
// all waves. float32 queries and weights enter as three bf16 parts, 3 products of
// bf16 where float32 ones take 16 times as long. 2048 tokens after 30 011, 32 and
// 8 heads of 128: 0.98 to 1.02 ms by card (1.02 to 1.07 PFLOP/s; over a bf16 cache
// 0.91 to 1.00); float32, 2048 after 8000, 8 and 4 heads of 64 / 128 / 256: 134 /
// 263 / 458 us (307 / 667 / 1250 over a float32 cache with float32 products).
// The values' writes have 2-way bank conflicts, a sixth of the LDS cycles; without
// them the time was the same.
//
// Few rows (decode steps, drafts): see below.
#include <hip/hip_runtime.h>

#include "paged_attn_core.h"
#include "paged_q4.h"

namespace rglru {
namespace paged {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

struct Attn4Args : AttnArgs {
  const uint8_t* ks;
  const uint8_t* vs;
};

// Eight values, the codes of `w` times `power`, as bf16 (NaN for a power that is an infinity).
__device__ __forceinline__ u32x4 values_of(uint32_t w, float power) {
  const u32x4 v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 0)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 1)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 2)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 3))};
  return v;
}

// Row j of a sequence in the cache, [n_pages, Hkv, page_size].
__device__ __forceinline__ int64_t cache_row(const AttnArgs& a, int32_t page, int hk, int32_t j) {
  const int64_t p = min(max(page, 0), a.n_pages - 1);
  return ((p * a.Hkv + hk) << a.lps) + (j & ((1 << a.lps) - 1));
}

// ---- many rows: the source of the tiles ----
template <typename E, int D>
struct Staged {
  typedef Attn4Args Args;
  typedef uint16_t Cache;
  using P = Wide<E, D, uint16_t>;
  using L = Tile<uint16_t, D>;
  static constexpr int kMine = P::kKeys / P::kWaves;         // rows of a wave
  static constexpr int kWords = kMine * D / 2 / 64 / 4;      // of a lane: 8 codes each
  static constexpr int kLanes = D / 8 / kWords;              // of a row
  static_assert(kWords >= 1 && 32 % (8 * kWords) == 0 && kMine * kLanes == 64, "a lane's codes are of one block");
  typedef uint32_t words __attribute__((ext_vector_type(kWords)));
  words k, v;
  uint32_t kb, vb;

  __device__ __forceinline__ void fetch(const Attn4Args& a, int32_t page, int hk, int32_t j, int, uint32_t, int lane) {
    const int64_t at = cache_row(a, page, hk, j);
    k = *reinterpret_cast<const words*>(a.kc + at * (D / 2) + lane * (4 * kWords));
    v = *reinterpret_cast<const words*>(a.vc + at * (D / 2) + lane * (4 * kWords));
    kb = a.ks[at * (D / 32) + lane * kWords / 4];
    vb = a.vs[at * (D / 32) + lane * kWords / 4];
  }
  __device__ __forceinline__ void put(lds_u8* to, int row, int lane) {
    const int r = row + lane / kLanes, c = lane % kLanes * kWords;
    const float kp = __uint_as_float(kb << 23), vp = __uint_as_float(vb << 23);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      *(lds_u32x4*)(to + r * L::kRowBytes + ((c + i) ^ L::swz_k(r)) * 16) = values_of(k[i], kp);
      *(lds_u32x4*)(to + P::kTileBytes + r * L::kRowBytes + ((c + i) ^ L::swz_v(r)) * 16) = values_of(v[i], vp);
    }
  }
  __device__ __forceinline__ void arrived() {}
};

// ---- few rows: at most 32 per unit (decode steps, drafts) ----
//
// Bound by the bytes of the cache and next by the vector units, which turn codes
// into values: a key and a value of 128 elements cost 136 bytes and, at 16 rows,
// 7 vector instructions of a wave. A wave therefore holds 16 rows (two sets of
// them where there are more) as the columns of S^T = K Q^T in 16x16 products, and
// streams tiles of 64 keys of its own through LDS as they lie in memory, codes and
// scales. 64 decodes over up to 16k tokens, 32 and 8 heads of 128: 113 us and a
// join of 6 (5.1 TB/s; 5.6 over 260k tokens a sequence, 48 of the 113 us would be
// vector instructions alone). float32, 32 drafts over up to 4k tokens, 16 heads of
// 64: 30 us, of them 8 of start and end (3.8 TB/s at length: three weights to
// lower and three products where bf16 has one).
//
// S^T: lane (m, g) = (lane % 16, lane / 16) reads a quarter of row m of 16 keys,
// elements (D / 4) g on, and turns it into operands; the sum over the elements
// does not care for their order, so the queries are held in the same one. A block
// of keys lies within a lane's quarter (or two quarters within a block), so the
// power is an operand of the conversion.
//
// O^T = V^T P^T: the accumulator of S^T (keys 4g .. 4g + 3 of every 16, row m) is
// the operand of P^T up to the order of the keys. The transposing 4-bit LDS read
// hands a lane 16 keys of one column, in rows of the lane's own choice: 16 j + 4g + i.
// Their powers differ within a pair that the conversion takes, so V enters as codes
// and the powers go into the weights, a set of weights per block of columns: exact,
// and a value that is not finite stays out of the products of rows that do not see
// it, as codes are always finite. Scales of a tile that lie in different bands
// (see Band) are taken a band at a time, a pass over the values each.
constexpr int kFewKeys = 64, kFewOver = 1;

template <typename E>
struct Few {
  typedef Frag<uint16_t> type;   // of queries and weights
};
template <>
struct Few<float> {
  typedef Split type;
};

// Weight i of an operand: 0 for one of 0.
__device__ __forceinline__ uint32_t weight_bits(const Frag<uint16_t>& f, int i) { return f.w[i / 2] >> (16 * (i % 2)) & 0xFFFFu; }
__device__ __forceinline__ uint32_t weight_bits(const Split& f, int i) { return f.w[0][i / 2] >> (16 * (i % 2)) & 0xFFFFu; }

// top - 128 e, a pair at a time (the compiler takes a shift and a subtraction instead).
__device__ __forceinline__ u16x2 exponents_below(u16x2 e, uint32_t top) {
  uint32_t r;
  asm("v_pk_mad_u16 %0, %1, %2, %3" : "=v"(r) : "v"(__builtin_bit_cast(uint32_t, e)), "v"(0xFF80FF80u), "s"(top));
  return __builtin_bit_cast(u16x2, r);
}
// Word w of an operand with its exponents lowered, down to 0.
__device__ __forceinline__ uint32_t lower(uint32_t x, u16x2 less) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, x), less));
}
__device__ __forceinline__ void lower(Frag<uint16_t>& to, const Frag<uint16_t>& from, int w, u16x2 less) {
  to.w[w] = lower(from.w[w], less);
}
__device__ __forceinline__ void lower(Split& to, const Split& from, int w, u16x2 less) {
#pragma unroll
  for (int j = 0; j < 3; ++j) to.w[j][w] = lower(from.w[j][w], less);
}

__device__ __forceinline__ f32x4 mma16(const u32x4& a, const Frag<uint16_t>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b.w), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(const u32x4& a, const Split& b, f32x4 c) {
#pragma unroll
  for (int j = 2; j >= 0; --j)
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b.w[j]), c, 0, 0, 0);
  return c;
}

// A tile of 64 keys in LDS: codes of the keys, of the values, scales of the keys, of the values. Rows of kP pieces of 16 bytes;
// piece c of row r lies at column c ^ swz(r), so that the lanes that one LDS cycle serves fall on different banks: rows
// 16 j .. 16 j + 15 at one piece (keys), and rows 16 j + 4 g + i of one g at one piece (values).
template <typename E, int D, int kSets>
struct Narrow4 {
  static constexpr int kP = D / 32;
  static constexpr int kCodes = kFewKeys * D / 2, kScales = kFewKeys * kP;   // bytes
  static constexpr int kCodeLoads = kCodes / 1024, kScaleLoads = (kScales + 255) / 256, kLoads = kCodeLoads + kScaleLoads;
  static constexpr int kScaleBytes = kScaleLoads * 256;
  static constexpr int kTileBytes = 2 * kCodes + 2 * kScaleBytes;
  static constexpr int kLoadRows = 64 / kP;   // rows that one load of codes fetches
  static constexpr int kWaves = 4, kThreads = kWaves * 64, kStretches = kWaves;
  // Workgroups on a CU: as many as the registers of float32 allow without spills, one at D = 256. One set of bf16 (124 registers at
  // D = 64, 160 at 128) would fit another one, which was not timed.
  static constexpr int kGroups = D == 256 || (D == 128 && kSets == 2 && sizeof(E) == 4) ? 1 : D == 64 && kSets == 1 ? 3 : 2;
  // Two sets of float32 queries of 256 elements take 192 registers, which spills 469 of them; with their third parts in LDS 178
  // (32 x 32 rows over 4000 tokens, 4 key heads: 175 -> 116 us).
  static constexpr bool kRest = D == 256 && kSets == 2 && sizeof(E) == 4;
  static constexpr int kRestBytes = kRest ? kSets * (D / 32) * 1024 : 0;   // of a wave
  // Pages of 8 keys each, looked up two tiles ahead.
  static constexpr int kSegs = kFewKeys / kSeg, kRing = 2, kPageBytes = kRing * kSegs * 4;
  __device__ static constexpr int swz(int r) {
    return kP == 2 ? (r >> 3 ^ r >> 4) & 1 : kP == 4 ? (r >> 2 ^ r >> 4) & 3 : (r >> 1 & 1) | ((r >> 2 ^ r >> 4) & 3) << 1;
  }
};

// 64 lanes x 16 (4) bytes from each lane's address to LDS at `to`; see load_lds.
__device__ __forceinline__ void load_lds16(uint32_t to, const uint8_t* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory");
}
__device__ __forceinline__ void load_lds4(uint32_t to, const uint8_t* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "memory");
}

__device__ __forceinline__ float quarter_max(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quarter_sum(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Scales of values pass as weights' exponents, lowered from the top of a scale's band. The bands' borders are fixed, so what
// becomes of a key, and which keys are summed in one pass, depends on its own scale alone; borders drawn from a tile's largest scale
// would let a key that a row does not see change that row's rounding. Widths: a weight of 2^-80 is still a normal bf16 46 steps
// lower; the third part of a float32 one starts 2^-16 below it. The usual band is 104 to 149 in bf16 (blocks whose largest value is
// 7e-7 to 2e7) and 112 to 142 in float32 (2e-4 to 2e5). Tiles whose values lie across a border take a pass for each band: 64 x 1
// after 7999, 16 / 4 heads of 64 / 128 / 256, take 39 / 56 / 112 us in bf16 and 60 / 88 / 206 with two bands in every tile, 48 / 70 /
// 145 and 75 / 113 / 256 in float32.
template <typename E>
struct Band {
  static constexpr int kWidth = sizeof(E) == 2 ? 46 : 31, kFirst = sizeof(E) == 2 ? 11 : 18;   // kFirst: the lowest top
  static constexpr int kUsual = kFirst + (sizeof(E) == 2 ? 3 : 4) * kWidth;
  static constexpr int kLast = kFirst + (252 - kFirst) / kWidth * kWidth;   // the highest top below 252, which ends the last one
  // 253 and 254 stand alone: values with them may pass bf16.
  __device__ static constexpr int top(int e) {
    return e > 252 ? e : e > kLast ? 252 : e <= kFirst ? kFirst : (e - kFirst + kWidth - 1) / kWidth * kWidth + kFirst;
  }
  __device__ static constexpr int low(int top) {
    return top > 252 ? top : top > kLast ? kLast + 1 : top <= kFirst ? 0 : top - kWidth + 1;
  }
};

// Whether a key's scales (byte by byte) lie between `low` and `ref`.
template <int kP>
__device__ __forceinline__ bool within(const uint32_t* w, int ref, int low) {
  const u16x2 top = {uint16_t(ref), uint16_t(ref)};
  u16x2 far = 0;
#pragma unroll
  for (int i = 0; i < (kP + 3) / 4; ++i) {
    far = __builtin_elementwise_max(far, top - __builtin_bit_cast(u16x2, w[i] & 0x00FF00FFu));
    far = __builtin_elementwise_max(far, top - __builtin_bit_cast(u16x2, w[i] >> 8 & 0x00FF00FFu));
  }
  return max(far[0], far[1]) <= ref - low;
}

// kSets sets of 16 rows of one wave.
template <typename E, int D, int kSets>
struct Wave4 {
  using P = Narrow4<E, D, kSets>;
  using O = typename Few<E>::type;
  O q[kSets][D / 32];
  f32x4 o[kSets][D / 16];
  float m[kSets], c[kSets], l[kSets];   // as in Wave
  lds_u8* rest;   // this lane's third parts, 1024 bytes apart
  int32_t lo[kSets], hi[kSets];

  // This lane's share of the queries of its rows, elements (D / 4) g on, as they lie in memory ..
  struct Raw {
    u32x4 w[kSets][D / 32 * int(sizeof(E)) / 2];
  };
  __device__ __forceinline__ Raw queries(const AttnArgs& a, const Seq& s, int hk, int32_t rows, int lane) const {
    Raw raw;
#pragma unroll
    for (int z = 0; z < kSets; ++z) {
      const int32_t r = z * 16 + (lane & 15);
      const bool live = r < rows;
      const int32_t t = live ? r / a.group : 0, head = live ? r - t * a.group : 0;
      const u32x4* const src = reinterpret_cast<const u32x4*>(
          a.q + ((s.start + t) * a.q_stride + int64_t(hk * a.group + head) * D + (lane >> 4) * (D / 4)) * sizeof(E));
#pragma unroll
      for (int x = 0; x < D / 32 * int(sizeof(E)) / 2; ++x) {
        raw.w[z][x] = 0;
        if (live) raw.w[z][x] = src[x];
      }
    }
    return raw;
  }
  // .. and as operands.
  __device__ __forceinline__ void start(const AttnArgs& a, const Seq& s, const Raw& raw, int32_t rows, int lane) {
    const uint32_t keep = a.q_sign == 0 ? 0u : ~0u, flip = a.q_sign < 0 ? O::kSigns : 0u;
#pragma unroll
    for (int z = 0; z < kSets; ++z) {
      const int32_t r = z * 16 + (lane & 15);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        if constexpr (sizeof(E) == 2) q[z][x].w = raw.w[z][x];
        else q[z][x] = split_query(raw.w[z][2 * x], raw.w[z][2 * x + 1]);
        if (a.q_sign <= 0) set_bits(q[z][x], keep, flip);
        if constexpr (P::kRest) *(lds_u32x4*)(rest + (z * (D / 32) + x) * 1024) = q[z][x].w[2];
      }
#pragma unroll
      for (int x = 0; x < D / 16; ++x) o[z][x] = 0.0f;
      m[z] = c[z] = -INFINITY;
      l[z] = 0.0f;
      hi[z] = r < rows ? max(s.kv - s.fresh + r / a.group, -1) : -1;
      lo[z] = a.window > 0 ? max(hi[z] - a.window + 1, 0) : 0;
    }
  }

  __device__ __forceinline__ O query(int z, int x) const {
    O f = q[z][x];
    if constexpr (P::kRest) f.w[2] = *(const lds_u32x4*)(rest + (z * (D / 32) + x) * 1024);
    return f;
  }

  // A lane's share of keys 16 j + lane % 16: codes and powers.
  struct Keys {
    uint32_t w[D / 32];
    float power[(D + 127) / 128];
  };
  // Where a lane's share of keys 0 .. 15 lies in a tile; that of keys 16 j on lies at an XOR of j, as swz is linear over XOR.
  __device__ __forceinline__ static int keys_at(int lane) {
    const int r = lane & 15, g = lane >> 4;
    if constexpr (D == 64) return r * (D / 2) + ((g >> 1) ^ P::swz(r)) * 16 + (g & 1) * 8;
    else return r * (D / 2) + ((g * (D / 128)) ^ P::swz(r)) * 16;
  }
  __device__ __forceinline__ static Keys keys_of(const lds_u8* codes, const lds_u8* scales, int j, int at, int lane) {
    const int from = (at ^ (P::swz(16 * j) * 16)) + 16 * j * (D / 2), g = lane >> 4;
    const lds_u8* const sc = scales + (16 * j + (lane & 15)) * P::kP;
    Keys k;
    if constexpr (D == 64) {
      const u32x2 x = *(const __attribute__((address_space(3))) u32x2*)(codes + from);
      k.w[0] = x[0], k.w[1] = x[1];
      k.power[0] = __uint_as_float(uint32_t(sc[g >> 1]) << 23);
    } else {
#pragma unroll
      for (int h = 0; h < D / 128; ++h) {
        const u32x4 x = *(const lds_u32x4*)(codes + (from ^ (h * 16)));
#pragma unroll
        for (int i = 0; i < 4; ++i) k.w[4 * h + i] = x[i];
        k.power[h] = __uint_as_float(uint32_t(sc[g * (D / 128) + h]) << 23);
      }
    }
    return k;
  }

  // Scores of the 64 keys in LDS: s[z][j] are keys 16 j + 4 g .. of the tile.
  __device__ __forceinline__ void scores(const lds_u8* codes, const lds_u8* scales, int lane, f32x4 (*s)[4]) const {
    int at = keys_at(lane);
    fresh_value(at);
    Keys next = keys_of(codes, scales, 0, at, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const Keys now = next;
      if (j < 3) next = keys_of(codes, scales, j + 1, at, lane);
#pragma unroll
      for (int z = 0; z < kSets; ++z) s[z][j] = 0.0f;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const u32x4 k = values_of(now.w[x], now.power[x / 4]);
#pragma unroll
        for (int z = 0; z < kSets; ++z) s[z][j] = mma16(k, query(z, x), s[z][j]);
      }
      order();
    }
  }

  // Turns the scores of set z into weights; `full`: every row of the wave sees all 64 keys.
  __device__ __forceinline__ void weights(float scale2, int z, f32x4* s, int32_t kv0, bool full, int lane) {
    const int g = lane >> 4;
    if (!full) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t key = kv0 + 16 * j + 4 * g + i;
          if (key < lo[z] || key > hi[z]) s[j][i] = -INFINITY;
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[j][i]);
    top = quarter_max(top);
    // the wave branches together, each row decides for itself: what other rows see must not change its bits
    const bool grow = top * scale2 > c[z] + kSlack;
    if (__any(grow)) {
      const float m_new = grow ? fmaxf(m[z], top) : m[z], c_new = m_new * scale2;
      const float keep = grow && c[z] != -INFINITY ? __builtin_amdgcn_exp2f(c[z] - c_new) : 1.0f;
      if (__any(keep != 1.0f)) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x) o[z][x] *= keep;
      }
      l[z] *= keep;
      m[z] = m_new;
      c[z] = grow ? c_new : c[z];
    }
    const float base = c[z] == -INFINITY ? 0.0f : c[z];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[j][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i], scale2, -base));
        sum += s[j][i];
      }
    l[z] += sum;
  }

  // The scales of keys 16 j + 4 g + i: byte i kP + b of sc[j].
  struct Scales {
    uint32_t w[4][P::kP];
  };
  __device__ __forceinline__ static Scales scales_of(const lds_u8* scales, int lane) {
    Scales sc;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const lds_u8* const at = scales + (16 * j + 4 * (lane >> 4)) * P::kP;
      if constexpr (P::kP == 2) {
        const u32x2 x = *(const __attribute__((address_space(3))) u32x2*)at;
        sc.w[j][0] = x[0], sc.w[j][1] = x[1];
      } else {
#pragma unroll
        for (int h = 0; h < P::kP / 4; ++h) {
          const u32x4 x = *(const lds_u32x4*)(at + 16 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) sc.w[j][4 * h + i] = x[i];
        }
      }
    }
    return sc;
  }

  // Codes of 16 keys in column 16 x + lane % 16; `at`: where the row lies whose codes this lane hands to the others.
  __device__ __forceinline__ static int rows_at(int lane) {
    const int i = lane & 15, r = 16 * (i >> 2) + 4 * (lane >> 4) + (i & 3);
    return r * (D / 2) + P::swz(r) * 16;
  }
  __device__ __forceinline__ static i32x2 column(const lds_u8* codes, int x, int at) {
    return __builtin_amdgcn_ds_read_tr4_b64_v2i32(
        (__attribute__((address_space(3))) i32x2*)(codes + ((at ^ (x / 2 * 16)) + x % 2 * 8)));
  }

  // The weights of 64 keys as operands.
  __device__ __forceinline__ static O operand(const f32x4* s) {
    const float w[8] = {s[0][0], s[0][1], s[0][2], s[0][3], s[1][0], s[1][1], s[1][2], s[1][3]};
    return pack_as<O, E>(w);
  }

  // Adds 64 weighted values to the output: the values as their codes times 2^(ref - 127), the weights (bf16, none negative)
  // times 2^(e - ref), subtracted from their exponents down to 0. For scales e of the band below ref; a weight beside a scale of 255
  // counts as 0.
  __device__ __forceinline__ void values(const lds_u8* codes, const lds_u8* scales, int ref, int lane, const O (*p)[2]) {
    const Scales sc = scales_of(scales, lane);
    int at = rows_at(lane);
    fresh_value(at);
    const float power = __uint_as_float(uint32_t(ref) << 23);
    const uint32_t top = uint32_t(ref << 7) * 0x10001u;
#pragma unroll
    for (int b = 0; b < P::kP; ++b) {
      const i32x2 c[2] = {column(codes, 2 * b, at), column(codes, 2 * b + 1, at)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        O f[kSets];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          // keys 2 (w % 2) and the next of subtile 2 h + w / 2
          const int j = 2 * h + w / 2, one = w % 2 * 2 * P::kP + b, two = one + P::kP;
          const u16x2 e = __builtin_bit_cast(u16x2, __builtin_amdgcn_perm(sc.w[j][two / 4], sc.w[j][one / 4],
                                                                          0x0C000C00u | uint32_t(4 + two % 4) << 16 | uint32_t(one % 4)));
          const u16x2 less = exponents_below(e, top);
#pragma unroll
          for (int z = 0; z < kSets; ++z) lower(f[z], p[z][h], w, less);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const u32x4 v = values_of(uint32_t(c[y][h]), power);
#pragma unroll
          for (int z = 0; z < kSets; ++z) o[z][2 * b + y] = mma16(v, f[z], o[z][2 * b + y]);
        }
      }
      order();
    }
  }

  // Blocks of values that are NaN make the rows that see them (with a weight above 0) NaN in their columns.
  __device__ __forceinline__ void mark(const lds_u8* scales, int lane, const O (*p)[2]) {
#pragma unroll
    for (int b = 0; b < P::kP; ++b)
#pragma unroll
      for (int z = 0; z < kSets; ++z) {
        uint32_t hit = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t byte = scales[(16 * (i / 4) + 4 * (lane >> 4) + i % 4) * P::kP + b];
          hit |= byte == 255u ? weight_bits(p[z][i / 8], i % 8) : 0u;
        }
        hit |= uint32_t(__shfl_xor(int(hit), 16));
        hit |= uint32_t(__shfl_xor(int(hit), 32));
        if (hit != 0) o[z][2 * b] = o[z][2 * b + 1] = __uint_as_float(0x7FC00000u);
        order();
      }
  }
};

__device__ __forceinline__ int32_t few_size(const AttnArgs& a, const Seq& s) {
  if (s.fresh == 0 || int64_t(s.fresh) * a.group > kNarrowRows) return 0;
  const Span x = span_of<kFewKeys>(a, s, 0, s.fresh * a.group - 1);
  return x.hi - x.lo + kFewOver;
}

// The kernel's arguments, read anew: what only the start and the end of a unit use takes no scalar registers in between.
__device__ __forceinline__ Attn4Args args_again() {
  auto* p = (const __attribute__((address_space(4))) Attn4Args*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const Attn4Args*)p;
}

template <typename E, int D, int kSets>
__global__ __launch_bounds__((Narrow4<E, D, kSets>::kThreads), (Narrow4<E, D, kSets>::kGroups)) void narrow4_kernel(Attn4Args a) {
  using P = Narrow4<E, D, kSets>;
  using W = Wave4<E, D, kSets>;
  __shared__ __align__(1024) unsigned char buf[P::kWaves * P::kTileBytes];
  __shared__ __align__(16) int32_t page_buf[P::kWaves * P::kRing * P::kSegs];
  __shared__ int64_t scan_part[P::kWaves];
  __shared__ Seq found[P::kWaves];
  __shared__ int32_t found_seq[P::kWaves];
  __shared__ int64_t found_rest[P::kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b0 = blockIdx.x * P::kWaves, b = b0 + wave;   // this workgroup's first stretch, this wave's
  if (b0 == a.narrow.grid) {
    list_row_tiles<Wide<E, D, uint16_t>, P::kThreads>(a, scan_part, a.sched, a.row_tiles, a.sched + 2 + a.max_tiles);
    return;
  }

  // Total length, then the sequences that hold the starts of the waves' stretches. Up to a sequence per thread both come of
  // one scan.
  Seq own = {0, 0, 0};
  int64_t total = 0, size = 0, upto = 0;
  for (int n0 = 0; n0 < a.N; n0 += P::kThreads) {
    int64_t sum;
    own = {0, 0, 0};
    if (n0 + tid < a.N) own = seq_of(a, n0 + tid);
    size = int64_t(few_size(a, own)) * a.Hkv;
    upto = block_scan<P::kThreads>(size, scan_part, sum);
    total += sum;
  }
  if (total == 0) return;
  const Line line(total, a.narrow.grid, 1);
  if (line.start(b0) >= total) return;
  int64_t found_before = 0;
  for (int n0 = 0;; n0 += P::kThreads) {
    int64_t sum = total;
    if (a.N > P::kThreads) {
      own = {0, 0, 0};
      if (n0 + tid < a.N) own = seq_of(a, n0 + tid);
      size = int64_t(few_size(a, own)) * a.Hkv;
      upto = found_before + block_scan<P::kThreads>(size, scan_part, sum);
    }
    for (int v = 0; v < P::kWaves; ++v) {
      const int64_t at = line.start(b0 + v);
      if (at >= upto - size && at < upto) {
        found[v] = own;
        found_seq[v] = n0 + tid;
        found_rest[v] = at - (upto - size);
      }
    }
    found_before += sum;
    if (line.start(b0 + P::kWaves - 1) < found_before || n0 + P::kThreads >= a.N) break;
  }
  __syncthreads();
  // From here on the waves go on by themselves.
  int64_t pos = line.start(b);
  const int64_t end = line.start(b + 1);
  if (pos >= end) return;
  int n = __builtin_amdgcn_readfirstlane(found_seq[wave]);
  int64_t rest = uniform(found_rest[wave]);   // position within the sequence's units
  Seq s = {__builtin_amdgcn_readfirstlane(found[wave].start), __builtin_amdgcn_readfirstlane(found[wave].fresh),
           __builtin_amdgcn_readfirstlane(found[wave].kv)};
  __shared__ __align__(16) unsigned char rest_buf[P::kWaves * P::kRestBytes + 16];
  W w;
  w.rest = (lds_u8*)rest_buf + wave * P::kRestBytes + lane * 16;
  lds_u8* const mine = (lds_u8*)buf + wave * P::kTileBytes;
  const uint32_t mine_at = uint32_t(uintptr_t(mine));
  lds_u8* const ring = (lds_u8*)page_buf + wave * P::kPageBytes;
  const uint32_t ring_at = uint32_t(uintptr_t(ring));
  // What a lane loads: of codes, 16 bytes of row lane / kP of a load; of scales, 4 bytes of a key (two keys at D = 64). Offsets
  // from the place of the tile's first key in its page, and bytes from page to page. A load's first row and a lane's have no
  // bit in common, so a page's mask and the swizzle apply to each.
  const int mask = (1 << a.lps) - 1, code_row = lane / P::kP, scale_key = lane * 4 / P::kP;
  const uint32_t code_page = uint32_t(a.Hkv << a.lps) * (D / 2), scale_page = uint32_t(a.Hkv << a.lps) * P::kP;
  int code_lane = (code_row & mask) * (D / 2) + (lane % P::kP ^ P::swz(code_row)) * 16;
  int scale_lane = (scale_key & mask) * P::kP + lane * 4 % P::kP;
  const int seqs = a.N, lps = a.lps, window = a.window, last_of_cache = a.n_pages - 1;
  const float scale2 = a.scale2;
  while (pos < end && n < seqs) {
    const Attn4Args before = args_again();
    const int32_t rows = int64_t(s.fresh) * before.group > kNarrowRows ? 0 : s.fresh * before.group;
    if (rows == 0) {
      if (++n < seqs) s = seq_of(before, n);
      continue;
    }
    const Span x = span_of<kFewKeys>(before, s, 0, rows - 1);
    const int32_t tiles = x.hi - x.lo, size = tiles + kFewOver;
    const int hk = __builtin_amdgcn_readfirstlane(int(rest / size));
    const int32_t in = int32_t(rest - int64_t(hk) * size);   // where this stretch enters the unit and leaves it
    const int32_t out = int32_t(min(int64_t(size), in + (end - pos)));
    if (out <= kFewOver) break;   // left to the next workgroup
    const int32_t t0 = max(in - kFewOver, 0), t1 = out - kFewOver;
    const int32_t* const row = before.table + int64_t(n) * before.width;
    const int32_t last_page = max((s.kv - 1) >> lps, 0);
    const typename W::Raw raw = w.queries(before, s, hk, rows, lane);

    // Asks for the pages of tile t, one for 8 keys.
    auto look_up = [&](int32_t t) {
      const int32_t j = (x.lo + t) * kFewKeys + lane * kSeg;
      if (lane < P::kSegs)
        load_lds4(ring_at + uint32_t((t - t0) % P::kRing * (P::kSegs * 4)),
                  reinterpret_cast<const uint8_t*>(row + min(j >> lps, last_page)));
    };
    // Where this lane's pieces of tile t lie, from the caches' starts.
    uint64_t code_at[P::kCodeLoads], scale_at[P::kScaleLoads];
    auto locate = [&](int32_t t) {
      const lds_u8* const pages = ring + (t - t0) % P::kRing * (P::kSegs * 4);
      auto page = [&](int key) {
        const int32_t p = *(const __attribute__((address_space(3))) int32_t*)(pages + key / kSeg * 4);
        return uint32_t(min(max(p, 0), last_of_cache));
      };
      // the tile's place in its page, where one holds more than a tile
      const uint32_t first = uint32_t(((hk << lps) + ((x.lo + t) * kFewKeys & mask)));
      fresh_value(code_lane);
      fresh_value(scale_lane);
#pragma unroll
      for (int i = 0; i < P::kCodeLoads; ++i) {
        const int r = i * P::kLoadRows;
        code_at[i] = uint64_t(page(r + code_row)) * code_page +
                     ((first + (r & mask)) * uint32_t(D / 2) + uint32_t(code_lane ^ (P::swz(r) * 16)));
      }
#pragma unroll
      for (int i = 0; i < P::kScaleLoads; ++i) {
        const int key = i * 256 / P::kP;
        scale_at[i] = uint64_t(page(key + scale_key % kFewKeys)) * scale_page + ((first + (key & mask)) * uint32_t(P::kP) + uint32_t(scale_lane));
      }
    };
    auto load = [&](const uint8_t* codes, const uint8_t* scales, uint32_t code_to, uint32_t scale_to) {
#pragma unroll
      for (int i = 0; i < P::kCodeLoads; ++i) load_lds16(code_to + i * 1024, codes + code_at[i]);
#pragma unroll
      for (int i = 0; i < P::kScaleLoads; ++i)
        if (i * 256 + lane * 4 < P::kScales) load_lds4(scale_to + i * 256, scales + scale_at[i]);
    };
    auto load_keys = [&]() {
      const Attn4Args now = args_again();
      load(now.kc, now.ks, mine_at, mine_at + 2 * P::kCodes);
    };
    auto load_values = [&]() {
      const Attn4Args now = args_again();
      load(now.vc, now.vs, mine_at + P::kCodes, mine_at + 2 * P::kCodes + P::kScaleBytes);
    };
#pragma unroll 1
    for (int i = 0; i < P::kRing; ++i) look_up(t0 + i);
    wait_loads<0>();   // the pages and the queries are there, and no store of the unit before is counted below
    locate(t0);
    load_keys();
    load_values();
    w.start(before, s, raw, rows, lane);
    int ref = Band<E>::kUsual, low = Band<E>::low(ref);
    for (int32_t t = t0; t < t1; ++t) {
      const bool next = t + 1 < t1;
      const int32_t kv0 = (x.lo + t) * kFewKeys;
      const bool full = kv0 + kFewKeys - 1 <= x.first && (window == 0 || kv0 > x.last - window);
      const lds_u8* const scales = mine + 2 * P::kCodes;
      f32x4 sc[kSets][4];
      typename W::O p[kSets][2];
      // Behind these keys these values are in flight; what the next tile is looked up with came before them.
      wait_loads<P::kLoads>();
      w.scores(mine, scales, lane, sc);
      if (next) {
        locate(t + 1);
        wait_reads();
        look_up(t + P::kRing);
        load_keys();
      }
#pragma unroll
      for (int z = 0; z < kSets; ++z) {
        w.weights(scale2, z, sc[z], kv0, full, lane);
        p[z][0] = W::operand(sc[z]);
        p[z][1] = W::operand(sc[z] + 2);
      }
      // behind these values: the keys just asked for
      if (next) wait_loads<P::kLoads>();
      else wait_loads<0>();
      // a key's scales per lane; what lies behind the last key is not looked at
      uint32_t own[(P::kP + 3) / 4];
#pragma unroll
      for (int i = 0; i < (P::kP + 3) / 4; ++i) {
        const lds_u8* const at = scales + P::kScaleBytes + lane * P::kP + 4 * i;
        if constexpr (P::kP == 2) own[i] = *(const __attribute__((address_space(3))) uint16_t*)at * 0x10001u;
        else own[i] = *(const __attribute__((address_space(3))) uint32_t*)at;
      }
      const bool there = kv0 + lane < s.kv;
      constexpr int kBytes = 4 * ((P::kP + 3) / 4);
      auto byte = [&](int i) { return own[i / 4] >> (8 * (i % 4)) & 255u; };
      auto largest = [&]() {   // of the bytes below 255
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kBytes; ++i) top = max(top, there && byte(i) < 255u ? byte(i) : 0u);
        for (int d = 32; d > 0; d /= 2) top = max(top, uint32_t(__shfl_xor(int(top), d)));
        return int(__builtin_amdgcn_readfirstlane(top));
      };
      auto next_band = [&]() {
        ref = Band<E>::top(largest());
        low = Band<E>::low(ref);
      };
      bool bands = __any(there && !within<P::kP>(own, ref, low));
      if (bands) {
        next_band();
        bands = __any(there && !within<P::kP>(own, ref, low));
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < kBytes; ++i) odd |= uint32_t(byte(i) == 255u);
        if (__any(there && odd)) w.mark(scales + P::kScaleBytes, lane, p);
      }
      for (;;) {
        bool more = false;
        if (bands) {
          // more than one band, or NaN: a band at a time, 255 for the others
          next_band();
          uint32_t now[kBytes / 4] = {}, left = 0;
#pragma unroll
          for (int i = 0; i < kBytes; ++i) {
            const bool in = int(byte(i)) <= ref && int(byte(i)) >= low;
            now[i / 4] |= (in ? byte(i) : 255u) << (8 * (i % 4));
            left |= uint32_t(!in && int(byte(i)) < low);
            if (in) own[i / 4] |= 255u << (8 * (i % 4));
          }
          more = __any(there && left);
#pragma unroll
          for (int i = 0; i < kBytes / 4; ++i) {
            lds_u8* const at = mine + 2 * P::kCodes + P::kScaleBytes + lane * P::kP + 4 * i;
            if constexpr (P::kP == 2) *(__attribute__((address_space(3))) uint16_t*)at = uint16_t(now[i]);
            else *(__attribute__((address_space(3))) uint32_t*)at = now[i];
          }
          wait_reads();
        }
        w.values(mine + P::kCodes, scales + P::kScaleBytes, ref, lane, p);
        if (!more) break;
      }
      if (next) {
        wait_reads();
        load_values();
      }
    }

    // Rows of a unit that lies in this stretch are finished here; those of a piece go to the join.
    const Attn4Args after = args_again();
    const int g = lane >> 4;
    const bool whole = t0 == 0 && t1 == tiles;
    float* const part = after.narrow.parts + int64_t(2 * b + (t0 == 0 ? 1 : 0)) * part_floats<D>(kNarrowRows);
#pragma unroll
    for (int z = 0; z < kSets; ++z) {
      const int r = z * 16 + (lane & 15);
      const float l = quarter_sum(w.l[z]);
      if (l != l && w.c[z] == -INFINITY) w.c[z] = 0.0f;   // all scores NaN: not a row that sees nothing
      if (r >= rows) continue;
      if (whole) {
        const bool none = w.c[z] == -INFINITY;
        const float inv = none ? 0.0f : 1.0f / l;
        const int64_t to = out_row(after, s, hk, r);
#pragma unroll
        for (int y = 0; y < D / 16; ++y) {
          const f32x4 v = none ? f32x4{0, 0, 0, 0} : w.o[z][y] * inv;
          store4<E>(after.o + (to * D + y * 16 + 4 * g) * sizeof(E), v[0], v[1], v[2], v[3]);
        }
        if (after.lse != nullptr && g == 0) after.lse[to] = none ? -INFINITY : (w.c[z] + log2f(l)) * kLn2;
      } else {
#pragma unroll
        for (int y = 0; y < D / 16; ++y) *reinterpret_cast<f32x4*>(part + r * D + y * 16 + 4 * g) = w.o[z][y];
        if (g == 0) {
          part[kNarrowRows * D + r] = w.c[z];
          part[kNarrowRows * (D + 1) + r] = l;
        }
      }
    }
    if (lane == 0 && t0 == 0) {   // the unit's first piece
      int32_t* const join = after.narrow.joins + 2 * (int64_t(n) * after.Hkv + hk);
      join[0] = whole ? 0 : int32_t(line.before(pos - in + size) - b);
      join[1] = b + 1;
    }
    pos += out - in;
    rest = out < size ? rest + (out - in) : (hk + 1 < after.Hkv ? int64_t(hk + 1) * size : 0);
    if (out == size && hk + 1 == after.Hkv && ++n < seqs) s = seq_of(after, n);
  }
}

// In a call that needs the wide kernel the other one takes the sequences of few rows where there are more than kFewSeqs
// sequences or this many (sequence of few rows, key head) pairs. 450 calls of a chunk of 200 or 1000 tokens and 1 to 15 single
// tokens, after 200 to 8000 tokens, 1 to 16 key heads, with bounds of 0 to no bound: the choice costs 1.3 to 1.7 % more than
// the better of the two in the mean (always both 19 to 62 %, no bound 1.4 to 8 %).
template <typename E, int D>
constexpr int kFewUnits4 = sizeof(E) == 4 || D == 64 ? 64 : 40;

// One set of rows where no unit has more than 16, else two: 32 x 16 rows over 4000 tokens, 4 key heads of 64 / 128 / 256, take
// 26 / 31 / 44 us with one and 28 / 34 / 54 with two in bf16, 30 / 37 / 56 and 36 / 49 / 163 in float32. 32 x 32 rows take 29 /
// 39 / 57 us with two and 62 / 75 / 122 in the wide kernel, 38 / 53 / 121 and 65 / 130 / 207 in float32.
template <typename E, int D>
Plan plan4_of(const rglru_paged_shape_t& s) {
  using W = Wide<E, D, uint16_t>;
  return most_rows(s) <= 16 ? plan_of<Narrow4<E, D, 1>, W, D>(s, kFewKeys, kFewUnits4<E, D>)
                            : plan_of<Narrow4<E, D, 2>, W, D>(s, kFewKeys, kFewUnits4<E, D>);
}

template <typename E, int D>
size_t bytes_of(const rglru_paged_shape_t& s) {
  // a call of fewer new tokens than the workspace was made for may run the kernel for few rows alone, with one or two sets
  const int32_t group = s.q_heads / s.kv_heads;
  size_t bytes = plan4_of<E, D>(s).bytes;
  for (int32_t rows : {16, kNarrowRows}) {
    rglru_paged_shape_t few = s;
    few.max_new = rows / group;
    if (few.max_new == 0 || (s.max_new > 0 && s.max_new < few.max_new)) continue;
    const size_t need = plan4_of<E, D>(few).bytes;
    if (need > bytes) bytes = need;
  }
  return bytes;
}

template <typename E, int D, int kSets>
void launch_narrow(const Attn4Args& a, const Plan& p, hipStream_t st) {
  using P = Narrow4<E, D, kSets>;
  narrow4_kernel<E, D, kSets><<<unsigned(p.narrow_grid / P::kStretches + p.wide), P::kThreads, 0, st>>>(a);
}

template <typename E, int D>
void launch(const rglru_paged_shape_t& s, Attn4Args a, uint8_t* workspace, hipStream_t st) {
  using W = Wide<E, D, uint16_t>;
  const Plan p = plan4_of<E, D>(s);
  lay_out(a, p, workspace);
  if (p.narrow) most_rows(s) <= 16 ? launch_narrow<E, D, 1>(a, p, st) : launch_narrow<E, D, 2>(a, p, st);
  if (p.wide) {
    if (!p.narrow && !p.own_list) sched_kernel<W><<<1, kSchedThreads, 0, st>>>(a);
    wide_kernel<E, D, Staged<E, D>><<<unsigned(p.wide_grid), W::kThreads, 0, st>>>(a);
  }
  join<E, D, W, true>(s, a, p, st);
}

}  // namespace
}  // namespace paged
}  // namespace rglru

using namespace rglru;

extern "C" size_t rglru_paged_attn_q4_workspace_bytes(const rglru_paged_shape_t* sp) {
  if (sp == nullptr || paged::check(*sp) != RGLRU_OK) return 0;
  return RGLRU_PAGED_DISPATCH(*sp, paged::bytes_of, *sp);
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
  paged::Attn4Args a;
  paged::set_args(a, s, cu_seqlens, kv_lens, block_table, q, k_codes, v_codes, o, lse);
  a.ks = k_scales;
  a.vs = v_scales;
  RGLRU_PAGED_DISPATCH(s, paged::launch, s, a, static_cast<uint8_t*>(workspace), static_cast<hipStream_t>(stream));
  return launch_status();
}
