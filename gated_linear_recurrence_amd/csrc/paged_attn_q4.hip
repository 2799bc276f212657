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
// bf16 where float32 ones take 16 times as long.
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
// Bound by the bytes of the cache and close behind by the vector units, which
// turn codes into values: a key and a value of 128 elements cost 136 bytes and,
// at 16 rows, some 8 vector instructions of a wave. A wave therefore holds 16 rows
// (two sets of them where there are more) as the columns of S^T = K Q^T in 16x16
// products, and streams tiles of 64 keys of its own through LDS as they lie in
// memory, codes and scales.
//
// S^T: lane (m, g) = (lane % 16, lane / 16) reads a quarter of row m of 16 keys,
// elements (D / 4) g on, and turns it into operands; the sum over the elements
// does not care for their order, so the queries are held in the same one. A block
// of keys lies within a lane's quarter (or two quarters within a block), so the power is an
// operand of the conversion.
//
// O^T = V^T P^T: the accumulator of S^T (keys 4g .. 4g + 3 of every 16, row m) is
// the operand of P^T up to the order of the keys. The transposing 4-bit LDS read
// hands a lane 16 keys of one column, in rows of the lane's own choice: 16 j + 4g + i.
// Their powers differ within a pair that the conversion takes, so V enters as codes and the powers go
// into the weights, a set of weights per block of columns: exact, and a value that is
// not finite stays out of the products of rows that do not see it, as codes are
// always finite.
constexpr int kFewKeys = 64, kFewOver = 4;

template <typename E>
struct Few {
  typedef Frag<uint16_t> type;   // of queries and weights
};
template <>
struct Few<float> {
  typedef Split type;
};

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
// piece c of row r lies at column c ^ swz(r), so that the lanes that one LDS cycle serves fall on different banks.
template <typename E, int D>
struct Narrow4 {
  static constexpr int kP = D / 32;
  static constexpr int kCodes = kFewKeys * D / 2, kScales = kFewKeys * kP;   // bytes
  static constexpr int kTileBytes = 2 * kCodes + 2 * ((kScales + 255) / 256 * 256);
  static constexpr int kCodeLoads = kCodes / 1024, kScaleLoads = (kScales + 255) / 256, kLoads = kCodeLoads + kScaleLoads;
  static constexpr int kScaleBytes = kScaleLoads * 256;
  static constexpr int kLoadRows = 64 / kP;   // rows that one load of codes fetches
  static constexpr int kWaves = 4, kThreads = kWaves * 64, kBuffers = 2;
  static constexpr int kGroups = D == 256 ? 1 : 2;   // workgroups on a CU
  __device__ static constexpr int swz_k(int r) { return r / (16 / kP) & (kP - 1); }
  __device__ static constexpr int swz_v(int r) {
    return kP == 8 ? (r >> 1 & 1) | (r >> 4 & 3) << 1 : r >> 4 & (kP - 1);
  }
};

// 64 lanes x 16 (4) bytes from each lane's address to LDS at `to`; see load_lds.
__device__ __forceinline__ void load_lds16(uint32_t to, const uint8_t* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory");
}
__device__ __forceinline__ void load_lds4(uint32_t to, const uint8_t* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "memory");
}

// v[i] of n, chosen by the lane: n is a power of two.
template <int n>
__device__ __forceinline__ int64_t choose(const int64_t* v, int i) {
  if constexpr (n == 1) {
    return v[0];
  } else {
    const int64_t lo = choose<n / 2>(v, i), hi = choose<n / 2>(v + n / 2, i);
    return i & (n / 2) ? hi : lo;
  }
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

// kSets sets of 16 rows of one wave.
template <typename E, int D, int kSets>
struct Wave4 {
  using P = Narrow4<E, D>;
  using O = typename Few<E>::type;
  O q[kSets][D / 32];
  f32x4 o[kSets][D / 16];
  float m[kSets], c[kSets], l[kSets];   // as in Wave
  int32_t lo[kSets], hi[kSets];

  // This lane's share of the queries of row r: elements (D / 4) g on.
  __device__ __forceinline__ void start(const AttnArgs& a, const Seq& s, int hk, int32_t rows, int lane) {
    const int g = lane >> 4;
    const uint32_t keep = a.q_sign == 0 ? 0u : ~0u, flip = a.q_sign < 0 ? O::kSigns : 0u;
#pragma unroll
    for (int z = 0; z < kSets; ++z) {
      const int32_t r = z * 16 + (lane & 15);
      const bool live = r < rows;
      const int32_t t = live ? r / a.group : 0, head = live ? r - t * a.group : 0;
      const u32x4* const src = reinterpret_cast<const u32x4*>(
          a.q + ((s.start + t) * a.q_stride + int64_t(hk * a.group + head) * D + g * (D / 4)) * sizeof(E));
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const u32x4 none = 0;
        if constexpr (sizeof(E) == 2) q[z][x].w = live ? src[x] : none;
        else q[z][x] = split_query(live ? src[2 * x] : none, live ? src[2 * x + 1] : none);
        if (a.q_sign <= 0) set_bits(q[z][x], keep, flip);
      }
#pragma unroll
      for (int x = 0; x < D / 16; ++x) o[z][x] = 0.0f;
      m[z] = c[z] = -INFINITY;
      l[z] = 0.0f;
      hi[z] = live ? max(s.kv - s.fresh + r / a.group, -1) : -1;
      lo[z] = a.window > 0 ? max(hi[z] - a.window + 1, 0) : 0;
    }
  }

  // Scores of the 64 keys in LDS: s[z][j] are keys 16 j + 4 g .. of the tile.
  __device__ __forceinline__ void scores(const lds_u8* codes, const lds_u8* scales, int lane, f32x4 (*s)[4]) const {
    const int row = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 16 * j + row;
      const lds_u8* const at = codes + r * (D / 2);
      uint32_t w[D / 32];
      float power[(D + 127) / 128];
      if constexpr (D == 64) {
        const u32x2 x = *(const __attribute__((address_space(3))) u32x2*)(at + ((g >> 1) ^ P::swz_k(r)) * 16 + (g & 1) * 8);
        w[0] = x[0], w[1] = x[1];
        power[0] = __uint_as_float(uint32_t(scales[r * P::kP + (g >> 1)]) << 23);
      } else {
#pragma unroll
        for (int h = 0; h < D / 128; ++h) {
          const u32x4 x = *(const lds_u32x4*)(at + ((g * (D / 128) + h) ^ P::swz_k(r)) * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[4 * h + i] = x[i];
          power[h] = __uint_as_float(uint32_t(scales[r * P::kP + g * (D / 128) + h]) << 23);
        }
      }
#pragma unroll
      for (int z = 0; z < kSets; ++z) s[z][j] = 0.0f;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const u32x4 k = values_of(w[x], power[x / 4]);
#pragma unroll
        for (int z = 0; z < kSets; ++z) s[z][j] = mma16(k, q[z][x], s[z][j]);
      }
    }
  }

  // Turns the scores of set z into weights; `full`: every row of the wave sees all 64 keys.
  __device__ __forceinline__ void weights(const AttnArgs& a, int z, f32x4* s, int32_t kv0, bool full, int lane) {
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
    const bool grow = top * a.scale2 > c[z] + kSlack;
    if (__any(grow)) {
      const float m_new = grow ? fmaxf(m[z], top) : m[z], c_new = m_new * a.scale2;
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
        s[j][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i], a.scale2, -base));
        sum += s[j][i];
      }
    l[z] += sum;
  }

  // Adds 64 weighted values to the output. kOdd: a block among them is NaN.
  template <bool kOdd>
  __device__ __forceinline__ void values(const lds_u8* codes, const lds_u8* scales, int lane, const f32x4 (*s)[4]) {
    const int row = lane & 15, g = lane >> 4;
    const int r = 16 * (row >> 2) + 4 * g + (row & 3);   // the row whose codes this lane hands to the others
    // the scales of keys 16 j + 4 g ..: 4 kP bytes each
    uint32_t sc[4][P::kP];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const lds_u8* const at = scales + (16 * j + 4 * g) * P::kP;
      if constexpr (P::kP == 2) {
        const u32x2 x = *(const __attribute__((address_space(3))) u32x2*)at;
        sc[j][0] = x[0], sc[j][1] = x[1];
      } else {
#pragma unroll
        for (int h = 0; h < P::kP / 4; ++h) {
          const u32x4 x = *(const lds_u32x4*)(at + 16 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[j][4 * h + i] = x[i];
        }
      }
    }
#pragma unroll
    for (int b = 0; b < P::kP; ++b) {
      float power[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int byte = i * P::kP + b;
          const uint32_t e = sc[j][byte / 4] >> (8 * (byte % 4)) & 255u;
          power[j][i] = __uint_as_float(e << 23);
          if (kOdd && e == 255u) power[j][i] = __uint_as_float(0x7FC00000u);
        }
      O p[kSets][2];
#pragma unroll
      for (int z = 0; z < kSets; ++z)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[8];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = s[z][2 * h + j][i];
              w[4 * j + i] = kOdd && x == 0.0f ? 0.0f : x * power[2 * h + j][i];
            }
          p[z][h] = pack_as<O, E>(w);
        }
#pragma unroll
      for (int x = 2 * b; x < 2 * b + 2; ++x) {
        const i32x2 w = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
            (__attribute__((address_space(3))) i32x2*)(codes + r * (D / 2) + ((x / 2) ^ P::swz_v(r)) * 16 + x % 2 * 8));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 v = values_of(uint32_t(w[h]), 1.0f);
#pragma unroll
          for (int z = 0; z < kSets; ++z) o[z][x] = mma16(v, p[z][h], o[z][x]);
        }
      }
    }
  }
};

__device__ __forceinline__ int32_t few_size(const AttnArgs& a, const Seq& s) {
  if (s.fresh == 0 || int64_t(s.fresh) * a.group > kNarrowRows) return 0;
  const Span x = span_of<kFewKeys>(a, s, 0, s.fresh * a.group - 1);
  return x.hi - x.lo + kFewOver;
}

template <typename E, int D, int kSets>
__global__ __launch_bounds__((Narrow4<E, D>::kThreads), (Narrow4<E, D>::kGroups)) void narrow4_kernel(Attn4Args a) {
  using P = Narrow4<E, D>;
  using W = Wave4<E, D, kSets>;
  __shared__ __align__(1024) unsigned char buf[P::kWaves * P::kBuffers * P::kTileBytes];
  __shared__ int64_t scan_part[P::kWaves];
  __shared__ Seq found;
  __shared__ int32_t found_seq;
  __shared__ int64_t found_rest;
  __shared__ float merge_c[P::kWaves][32], merge_l[P::kWaves][32];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = blockIdx.x;
  if (b == a.narrow.grid) {
    list_row_tiles<Wide<E, D, uint16_t>, P::kThreads>(a, scan_part, a.sched, a.row_tiles, a.sched + 2 + a.max_tiles);
    return;
  }

  // Total length, then the sequence that holds this stretch's start. Up to a sequence per thread both come of one scan.
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
      size = int64_t(few_size(a, own)) * a.Hkv;
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
  lds_u8* const mine = (lds_u8*)buf + wave * P::kBuffers * P::kTileBytes;
  const uint32_t mine_at = uint32_t(uintptr_t(mine));
  // what a lane loads: of codes, 16 bytes of row lane / kP of a load; of scales, 4 bytes of a key (two keys at D = 64)
  const int code_row = lane / P::kP, code_col = lane % P::kP;
  while (pos < end && n < a.N) {
    const int32_t rows = int64_t(s.fresh) * a.group > kNarrowRows ? 0 : s.fresh * a.group;
    if (rows == 0) {
      if (++n < a.N) s = seq_of(a, n);
      continue;
    }
    const Span x = span_of<kFewKeys>(a, s, 0, rows - 1);
    const int32_t tiles = x.hi - x.lo, size = tiles + kFewOver;
    const int hk = __builtin_amdgcn_readfirstlane(int(rest / size));
    const int32_t in = int32_t(rest - int64_t(hk) * size);   // where this stretch enters the unit and leaves it
    const int32_t out = int32_t(min(int64_t(size), in + (end - pos)));
    if (out <= kFewOver) break;   // left to the next workgroup
    const int32_t t0 = max(in - kFewOver, 0), t1 = out - kFewOver;
    const_i32* row = (const_i32*)(a.table + int64_t(n) * a.width);
    const int32_t last_page = max((s.kv - 1) >> a.lps, 0);
    w.start(a, s, hk, rows, lane);

    // the pages of the tile to load next are looked up one tile ahead: 8 rows lie in one page
    constexpr int kSegs = kFewKeys / kSeg, kW = P::kWaves;
    int32_t pages[kSegs];
    int64_t at[kSegs];   // rows of the cache
    auto look_up = [&](int32_t t) {
      const int32_t kv0 = __builtin_amdgcn_readfirstlane((x.lo + t) * kFewKeys);
#pragma unroll
      for (int i = 0; i < kSegs; ++i) pages[i] = seg_page(a, row, last_page, kv0 + i * kSeg);
    };
    auto locate = [&](int32_t t) {
      const int32_t kv0 = __builtin_amdgcn_readfirstlane((x.lo + t) * kFewKeys);
#pragma unroll
      for (int i = 0; i < kSegs; ++i) at[i] = cache_row(a, pages[i], hk, kv0 + i * kSeg);
    };
    auto load = [&](const uint8_t* codes, const uint8_t* scales, uint32_t code_to, uint32_t scale_to, bool values) {
      constexpr int kPer = P::kLoadRows / kSeg;   // segments of a load
#pragma unroll
      for (int i = 0; i < P::kCodeLoads; ++i) {
        const int r = i * P::kLoadRows + code_row;
        const int64_t first = choose<kPer>(at + i * kPer, code_row / kSeg);
        const int col = code_col ^ (values ? P::swz_v(r) : P::swz_k(r));
        load_lds16(code_to + i * 1024, codes + first * (D / 2) + (code_row % kSeg) * (D / 2) + col * 16);
      }
#pragma unroll
      for (int i = 0; i < P::kScaleLoads; ++i) {
        const int byte = i * 256 + lane * 4, key = byte / P::kP;
        constexpr int kOf = kSegs / P::kScaleLoads;
        const int64_t first = choose<kOf>(at + i * kOf, key / kSeg % kOf);
        if (byte < P::kScales) load_lds4(scale_to + i * 256, scales + first * P::kP + byte % (kSeg * P::kP));
      }
    };
    auto load_keys = [&](uint32_t to) { load(a.kc, a.ks, to, to + 2 * P::kCodes, false); };
    auto load_values = [&](uint32_t to) { load(a.vc, a.vs, to + P::kCodes, to + 2 * P::kCodes + P::kScaleBytes, true); };
    look_up(t0 + wave);
    wait_loads<0>();   // no store of the unit before is counted below
    uint32_t half = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
      if (t0 + wave + i * kW < t1) {
        locate(t0 + wave + i * kW);
        load_keys(mine_at + i * P::kTileBytes);
        load_values(mine_at + i * P::kTileBytes);
        look_up(t0 + wave + (i + 1) * kW);
      }
    for (int32_t t = t0 + wave; t < t1; t += kW) {
      const bool next = t + kW < t1, after = t + 2 * kW < t1;   // a further tile, and one for the buffer that this one leaves
      const int32_t kv0 = (x.lo + t) * kFewKeys;
      const bool full = kv0 + kFewKeys - 1 <= x.first && (a.window == 0 || kv0 > x.last - a.window);
      lds_u8* const tile = mine + half;
      const lds_u8* const scales = tile + 2 * P::kCodes;
      f32x4 sc[kSets][4];
      // behind these keys are in flight: these values and the next tile
      if (next) wait_loads<3 * P::kLoads>();
      else wait_loads<P::kLoads>();
      w.scores(tile, scales, lane, sc);
      if (after) {
        wait_reads();
        locate(t + 2 * kW);
        load_keys(mine_at + half);
      }
#pragma unroll
      for (int z = 0; z < kSets; ++z) w.weights(a, z, sc[z], kv0, full, lane);
      // behind these values: the keys just asked for and the next tile
      if (after) wait_loads<3 * P::kLoads>();
      else if (next) wait_loads<2 * P::kLoads>();
      else wait_loads<0>();
      // whether a block among the values is NaN: a key's scales per lane
      uint32_t nan = 0;
#pragma unroll
      for (int i = 0; i < (P::kP + 3) / 4; ++i) {
        uint32_t z;
        if constexpr (P::kP == 2) z = *(const __attribute__((address_space(3))) uint16_t*)(scales + P::kScaleBytes + lane * 2);
        else z = *(const __attribute__((address_space(3))) uint32_t*)(scales + P::kScaleBytes + lane * P::kP + 4 * i);
        nan |= ((z & 0x7F7F7F7Fu) + 0x01010101u) & z;
      }
      if (__any((nan & 0x80808080u) != 0)) w.template values<true>(tile + P::kCodes, scales + P::kScaleBytes, lane, sc);
      else w.template values<false>(tile + P::kCodes, scales + P::kScaleBytes, lane, sc);
      if (after) {
        wait_reads();
        load_values(mine_at + half);
        look_up(t + 3 * kW);
      }
      half ^= P::kTileBytes;
    }

    // The waves merge: maxima and sums first, then every thread sums some columns over the waves.
    const int q = lane & 15, g = lane >> 4;
    __syncthreads();   // the buffers are free
    float* const sums = reinterpret_cast<float*>(buf);
#pragma unroll
    for (int z = 0; z < kSets; ++z) {
      const float l_all = quarter_sum(w.l[z]);
      if (l_all != l_all && w.c[z] == -INFINITY) w.c[z] = 0.0f;   // all scores NaN: not a row that sees nothing
      if (g == 0) {
        merge_c[wave][z * 16 + q] = w.c[z];
        merge_l[wave][z * 16 + q] = l_all;
      }
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == tiles;
    float* const part = a.narrow.parts + int64_t(2 * b + (t0 == 0 ? 1 : 0)) * part_floats<D>(kNarrowRows);
    // half of the columns at a time, in the buffers of the tiles
#pragma unroll
    for (int x0 = 0; x0 < D; x0 += D / 2) {
      constexpr int kC = D / 2, kRow = kC + 4;   // 4 floats against bank conflicts
      static_assert(P::kWaves * 32 * kRow * 4 <= int(sizeof(buf)), "merge buffer");
#pragma unroll
      for (int z = 0; z < kSets; ++z)
        if (z * 16 + q < rows) {
#pragma unroll
          for (int y = 0; y < kC / 16; ++y)
            *reinterpret_cast<f32x4*>(sums + (wave * 32 + z * 16 + q) * kRow + y * 16 + 4 * g) = w.o[z][x0 / 16 + y];
        }
      __syncthreads();
      for (int e = tid; e < rows * (kC / 4); e += P::kThreads) {
        const int qq = e / (kC / 4), d = (e % (kC / 4)) * 4;
        float top = -INFINITY;
        for (int v = 0; v < P::kWaves; ++v) top = fmaxf(top, merge_c[v][qq]);
        const float base = top == -INFINITY ? 0.0f : top;
        f32x4 acc = 0.0f;
        float l = 0.0f;
        for (int v = 0; v < P::kWaves; ++v) {
          // a part without weights counts too, by a factor of 0: what it saw may have been NaN
          const float f = __builtin_amdgcn_exp2f(merge_c[v][qq] - base);
          acc += f * *reinterpret_cast<const f32x4*>(sums + (v * 32 + qq) * kRow + d);
          l += f * merge_l[v][qq];
        }
        const int col = x0 + d;
        if (whole) {
          const float inv = top == -INFINITY ? 0.0f : 1.0f / l;
          if (top == -INFINITY) acc = 0.0f;
          const int64_t r = out_row(a, s, hk, qq);
          store4<E>(a.o + (r * D + col) * sizeof(E), acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
          if (a.lse != nullptr && col == 0) a.lse[r] = top == -INFINITY ? -INFINITY : (top + log2f(l)) * kLn2;
        } else {
          *reinterpret_cast<f32x4*>(part + qq * D + col) = acc;
          if (col == 0) {
            part[kNarrowRows * D + qq] = top;
            part[kNarrowRows * (D + 1) + qq] = l;
          }
        }
      }
      __syncthreads();
    }
    if (tid == 0 && t0 > 0 && line.start(b - 1) <= pos - in + kFewOver) {
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

// In a call that needs the wide kernel the other one takes the sequences of few rows where there are more than kFewSeqs
// sequences or this many (sequence of few rows, key head) pairs.
constexpr int kFewUnits4 = 64;

template <typename E, int D>
Plan plan4_of(const rglru_paged_shape_t& s) {
  return plan_of<Narrow4<E, D>, Wide<E, D, uint16_t>, D>(s, kFewKeys, kFewUnits4);
}

template <typename E, int D>
size_t bytes_of(const rglru_paged_shape_t& s) {
  return plan4_of<E, D>(s).bytes;
}

template <typename E, int D>
void launch(const rglru_paged_shape_t& s, Attn4Args a, uint8_t* workspace, hipStream_t st) {
  using W = Wide<E, D, uint16_t>;
  const Plan p = plan4_of<E, D>(s);
  lay_out(a, p, workspace);
  if (p.narrow) {
    const unsigned grid = unsigned(p.narrow_grid + p.wide);
    if (most_rows(s) <= 16) narrow4_kernel<E, D, 1><<<grid, Narrow4<E, D>::kThreads, 0, st>>>(a);
    else narrow4_kernel<E, D, 2><<<grid, Narrow4<E, D>::kThreads, 0, st>>>(a);
  }
  if (p.wide) {
    if (!p.narrow && !p.own_list) sched_kernel<W><<<1, kSchedThreads, 0, st>>>(a);
    wide_kernel<E, D, Staged<E, D>><<<unsigned(p.wide_grid), W::kThreads, 0, st>>>(a);
  }
  join<E, D, W>(s, a, p, st);
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
