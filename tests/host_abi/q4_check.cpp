// Host-side checks of the 4-bit cache's and the page pool's entry points, built with
// AddressSanitizer and UndefinedBehaviorSanitizer around the library's host
// code (host-only compile: no kernel runs): the size queries over ordinary and extreme
// shapes, and every refusal, which must come before anything is launched.
// Prints one line per failed expectation and exits nonzero if any failed.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "page_pool.h"
#include "paged_q4.h"

static int g_fail = 0;

#define EXPECT(cond)                                                   \
  do {                                                                 \
    if (!(cond)) {                                                     \
      std::printf("FAIL line %d: %s\n", __LINE__, #cond);              \
      ++g_fail;                                                        \
    }                                                                  \
  } while (0)

static const rglru_status_t kInvalid = RGLRU_ERR_INVALID_ARGUMENT;

static rglru_paged_shape_t shape() {
  rglru_paged_shape_t s = {};
  s.n_tokens = 40;
  s.n_pages = 100;
  s.n_seqs = 3;
  s.max_pages = 30;
  s.page_size = 16;
  s.q_heads = 8;
  s.kv_heads = 2;
  s.head_dim = 128;
  s.io_dtype = RGLRU_IO_BF16;
  s.scale = 0.1f;
  return s;
}

template <typename T>
static T* as(uintptr_t at) {  // never dereferenced: every call here is refused or has nothing to do
  return reinterpret_cast<T*>(at);
}
static uintptr_t at(int i) { return (uintptr_t(i) + 1) << 36; }

// Every entry point with argument `moved` at `to` and each other one at a place of its own.
static rglru_status_t attn(const rglru_paged_shape_t* s, int moved = -1, uintptr_t to = 0, size_t bytes = ~size_t(0)) {
  uintptr_t p[11];
  for (int i = 0; i < 11; ++i) p[i] = i == moved ? to : at(i);
  return rglru_paged_attn_q4_fwd(s, as<int32_t>(p[0]), as<int32_t>(p[1]), as<int32_t>(p[2]), as<void>(p[3]), as<uint8_t>(p[4]),
                                 as<uint8_t>(p[5]), as<uint8_t>(p[6]), as<uint8_t>(p[7]), as<void>(p[8]), as<float>(p[9]),
                                 as<void>(p[10]), bytes == ~size_t(0) ? rglru_paged_attn_q4_workspace_bytes(s) : bytes, nullptr);
}
static rglru_status_t write(const rglru_paged_shape_t* s, int moved = -1, uintptr_t to = 0) {
  uintptr_t p[7];
  for (int i = 0; i < 7; ++i) p[i] = i == moved ? to : at(i);
  return rglru_paged_kv_write_q4(s, as<void>(p[0]), as<void>(p[1]), as<uint8_t>(p[2]), as<uint8_t>(p[3]), as<uint8_t>(p[4]),
                                 as<uint8_t>(p[5]), as<int32_t>(p[6]), nullptr);
}
static rglru_status_t read(const rglru_paged_shape_t* s, int moved = -1, uintptr_t to = 0) {
  uintptr_t p[7];
  for (int i = 0; i < 7; ++i) p[i] = i == moved ? to : at(i);
  return rglru_paged_kv_read_q4(s, as<uint8_t>(p[2]), as<uint8_t>(p[3]), as<uint8_t>(p[4]), as<uint8_t>(p[5]), as<int32_t>(p[6]),
                                as<void>(p[0]), as<void>(p[1]), nullptr);
}
static rglru_status_t fork(const rglru_paged_shape_t* s, int moved = -1, uintptr_t to = 0) {
  uintptr_t p[12];
  for (int i = 0; i < 12; ++i) p[i] = i == moved ? to : at(i);
  return rglru_page_fork(s, as<int32_t>(p[0]), as<int32_t>(p[1]), as<int32_t>(p[2]), as<int32_t>(p[5]), as<int32_t>(p[6]),
                         as<int32_t>(p[3]), as<int32_t>(p[4]), as<int32_t>(p[7]), as<int32_t>(p[8]), as<int32_t>(p[9]),
                         as<int32_t>(p[10]), as<int32_t>(p[11]), nullptr);
}
static rglru_status_t release(const rglru_paged_shape_t* s, int moved = -1, uintptr_t to = 0, size_t bytes = 1 << 20) {
  uintptr_t p[9];
  for (int i = 0; i < 9; ++i) p[i] = i == moved ? to : at(i);
  return rglru_page_free(s, as<int32_t>(p[0]), as<int32_t>(p[1]), as<int32_t>(p[2]), as<int32_t>(p[4]), as<int32_t>(p[5]),
                         as<int32_t>(p[3]), as<int32_t>(p[6]), as<int32_t>(p[7]), as<void>(p[8]), bytes, nullptr);
}
static rglru_status_t compact(const rglru_paged_shape_t* s, int moved = -1, uintptr_t to = 0, int64_t keep = 50, size_t bytes = 1 << 20) {
  uintptr_t p[13];
  for (int i = 0; i < 13; ++i) p[i] = i == moved ? to : at(i);
  return rglru_page_compact(s, keep, as<int32_t>(p[0]), as<int32_t>(p[1]), as<int32_t>(p[2]), as<int32_t>(p[3]), as<int32_t>(p[4]),
                            as<int32_t>(p[5]), as<int32_t>(p[6]), as<int32_t>(p[7]), as<int32_t>(p[8]), as<int32_t>(p[9]),
                            as<int32_t>(p[10]), as<int32_t>(p[11]), as<void>(p[12]), bytes, nullptr);
}

int main() {
  const int64_t big64[] = {-1, std::numeric_limits<int64_t>::min(), std::numeric_limits<int64_t>::max(), int64_t(1) << 31,
                           int64_t(1) << 40};
  const int32_t big32[] = {-1, std::numeric_limits<int32_t>::min(), std::numeric_limits<int32_t>::max()};
  EXPECT(rglru_paged_attn_q4_workspace_bytes(nullptr) == 0 && rglru_page_free_workspace_bytes(nullptr) == 0 &&
         rglru_page_compact_workspace_bytes(nullptr) == 0);
  EXPECT(attn(nullptr, -1, 0, 0) == kInvalid && write(nullptr) == kInvalid && read(nullptr) == kInvalid && fork(nullptr) == kInvalid &&
         release(nullptr) == kInvalid && compact(nullptr) == kInvalid);

  // sizes: nonzero, a multiple of what they are aligned to
  rglru_paged_shape_t s = shape();
  for (int io : {0, 1})
    for (int d : {64, 128, 256})
      for (int group : {1, 5, 16, 300})
        for (int64_t t : {int64_t(0), int64_t(1), int64_t(7), int64_t(5000), int64_t(1) << 21}) {
          s = shape();
          s.io_dtype = io;
          s.head_dim = d;
          s.q_heads = s.kv_heads * group;
          s.n_tokens = t;
          const size_t a = rglru_paged_attn_q4_workspace_bytes(&s);
          EXPECT(a > 0 && a % 256 == 0 && a < (size_t(1) << 32));
        }
  s = shape();
  s.n_pages = (int64_t(1) << 31) / 8 - 1;
  s.page_size = 8;
  s.max_pages = ((int64_t(1) << 31) - (1 << 16)) / 8;
  s.n_seqs = 1 << 16;
  s.q_heads = s.kv_heads = 1;
  s.n_tokens = (int64_t(1) << 31) - (1 << 16);
  EXPECT(rglru_paged_attn_q4_workspace_bytes(&s) > 0);
  EXPECT(rglru_page_free_workspace_bytes(&s) % 16 == 0 && rglru_page_free_workspace_bytes(&s) >= 16);
  EXPECT(rglru_page_compact_workspace_bytes(&s) % 16 == 0 && rglru_page_compact_workspace_bytes(&s) > size_t(s.n_pages) * 6);
  s.n_tokens += 1;
  EXPECT(rglru_paged_attn_q4_workspace_bytes(&s) == 0);

  // every refused shape, by who reads the field
  enum { A = 1, W = 2, P = 4 };   // attention, write and read, pool
  auto bad = [](auto change, int who) {
    rglru_paged_shape_t b = shape();
    change(b);
    if (who & A) EXPECT(attn(&b, -1, 0, 1 << 30) == kInvalid && rglru_paged_attn_q4_workspace_bytes(&b) == 0);
    if (who & W) EXPECT(write(&b) == kInvalid && (read(&b) == kInvalid || b.kv_stride != 0));
    if (who & P) {
      EXPECT(fork(&b) == kInvalid && release(&b) == kInvalid && compact(&b) == kInvalid);
      EXPECT(rglru_page_free_workspace_bytes(&b) == 0 && rglru_page_compact_workspace_bytes(&b) == 0);
    }
  };
  for (int64_t v : big64) {
    bad([v](rglru_paged_shape_t& b) { b.n_tokens = v; }, A | W);
    bad([v](rglru_paged_shape_t& b) { b.n_pages = v; }, A | W | P);
    if (v != (int64_t(1) << 31) - 1) bad([v](rglru_paged_shape_t& b) { b.q_stride = v < 0 ? v : int64_t(1) << 40; }, A);
    bad([v](rglru_paged_shape_t& b) { b.kv_stride = v < 0 ? v : int64_t(1) << 40; }, W);
  }
  for (int32_t v : big32) {
    bad([v](rglru_paged_shape_t& b) { b.n_seqs = v; }, A | P);
    bad([v](rglru_paged_shape_t& b) { b.max_pages = v; }, A | P);
    bad([v](rglru_paged_shape_t& b) { b.page_size = v; }, A | W | P);
    bad([v](rglru_paged_shape_t& b) { b.q_heads = v; }, A);
    bad([v](rglru_paged_shape_t& b) { b.kv_heads = v; }, A | W);
    bad([v](rglru_paged_shape_t& b) { b.head_dim = v; }, A | W);
    bad([v](rglru_paged_shape_t& b) { b.io_dtype = v; }, A | W);
    if (v < 0) {
      bad([v](rglru_paged_shape_t& b) { b.max_new = v; }, A);
      bad([v](rglru_paged_shape_t& b) { b.window = v; }, A);
    }
  }
  bad([](rglru_paged_shape_t& b) { b.n_pages = 0; }, A | W | P);
  bad([](rglru_paged_shape_t& b) { b.n_seqs = 0; }, A | P);
  bad([](rglru_paged_shape_t& b) { b.n_seqs = (1 << 16) + 1; }, A | P);
  bad([](rglru_paged_shape_t& b) { b.max_pages = 0; }, A | P);
  for (int p : {0, 1, 4, 7, 12, 2048}) bad([p](rglru_paged_shape_t& b) { b.page_size = p; }, A | W | P);
  bad([](rglru_paged_shape_t& b) { b.q_heads = 7; }, A);
  bad([](rglru_paged_shape_t& b) { b.head_dim = 0; }, A | W);
  bad([](rglru_paged_shape_t& b) { b.scale = std::numeric_limits<float>::quiet_NaN(); }, A);
  bad([](rglru_paged_shape_t& b) { b.scale = 3e38f; }, A);
  bad([](rglru_paged_shape_t& b) { b.q_stride = 8 * 128 - 8; }, A);
  bad([](rglru_paged_shape_t& b) { b.kv_stride = 2 * 128 - 8; }, W);
  // 2^36 - 2^12 bytes of keys
  s = shape();
  s.io_dtype = RGLRU_IO_F32;
  s.kv_heads = 1 << 14;
  s.n_tokens = (int64_t(1) << 31) - 1;
  EXPECT(write(&s) == kInvalid && read(&s) == kInvalid);

  // unsupported, misaligned, too small, null
  s = shape();
  s.head_dim = 96;
  EXPECT(attn(&s, -1, 0, 1 << 20) == RGLRU_ERR_UNSUPPORTED && rglru_paged_attn_q4_workspace_bytes(&s) == 0);
  s.head_dim = 48;
  EXPECT(write(&s) == RGLRU_ERR_UNSUPPORTED && read(&s) == RGLRU_ERR_UNSUPPORTED);
  s = shape();
  s.q_stride = 8 * 128 + 4;
  EXPECT(attn(&s) == RGLRU_ERR_MISALIGNED);
  s = shape();
  s.kv_stride = 2 * 128 + 4;
  EXPECT(write(&s) == RGLRU_ERR_MISALIGNED);
  s = shape();
  for (int i = 0; i < 11; ++i) {
    EXPECT(attn(&s, i, at(i) + 2) == RGLRU_ERR_MISALIGNED);
    if (i != 9) EXPECT(attn(&s, i, 0) == kInvalid);   // lse may be NULL
  }
  for (int i : {3, 4, 5, 6, 7, 8}) EXPECT(attn(&s, i, at(i) + 8) == RGLRU_ERR_MISALIGNED);
  EXPECT(attn(&s, 10, at(10) + 128) == RGLRU_ERR_MISALIGNED);
  EXPECT(attn(&s, -1, 0, rglru_paged_attn_q4_workspace_bytes(&s) - 1) == RGLRU_ERR_WORKSPACE_TOO_SMALL);
  for (int i = 0; i < 7; ++i) {
    EXPECT(write(&s, i, at(i) + 2) == RGLRU_ERR_MISALIGNED && read(&s, i, at(i) + 2) == RGLRU_ERR_MISALIGNED);
    if (i < 6) EXPECT(write(&s, i, at(i) + 8) == RGLRU_ERR_MISALIGNED && read(&s, i, at(i) + 8) == RGLRU_ERR_MISALIGNED);
    EXPECT(write(&s, i, 0) == kInvalid && read(&s, i, 0) == kInvalid);
  }
  for (int i = 0; i < 12; ++i) {
    EXPECT(fork(&s, i, at(i) + 2) == RGLRU_ERR_MISALIGNED);
    if (i != 2) EXPECT(fork(&s, i, 0) == kInvalid);   // held_lens may be NULL
  }
  for (int i = 0; i < 9; ++i) EXPECT(release(&s, i, at(i) + 2) == RGLRU_ERR_MISALIGNED && release(&s, i, 0) == kInvalid);
  EXPECT(release(&s, 8, at(8) + 8) == RGLRU_ERR_MISALIGNED && release(&s, -1, 0, 8) == RGLRU_ERR_WORKSPACE_TOO_SMALL);
  for (int i = 0; i < 13; ++i) EXPECT(compact(&s, i, at(i) + 2) == RGLRU_ERR_MISALIGNED && compact(&s, i, 0) == kInvalid);
  EXPECT(compact(&s, 12, at(12) + 8) == RGLRU_ERR_MISALIGNED);
  EXPECT(compact(&s, -1, 0, 50, rglru_page_compact_workspace_bytes(&s) - 1) == RGLRU_ERR_WORKSPACE_TOO_SMALL);
  for (int64_t keep : {int64_t(-1), int64_t(101), std::numeric_limits<int64_t>::max(), std::numeric_limits<int64_t>::min()})
    EXPECT(compact(&s, -1, 0, keep) == kInvalid);

  // outputs that overlap an input or each other, by a whole array or by its last bytes
  const int64_t o_size = s.n_tokens * s.q_heads * s.head_dim * 2, codes = s.n_pages * s.page_size * s.kv_heads * s.head_dim / 2;
  for (int out = 8; out < 11; ++out)
    for (int other = 0; other < 11; ++other)
      if (other != out) EXPECT(attn(&s, out, at(other)) == kInvalid);
  EXPECT(attn(&s, 3, at(8) + o_size - 16) == kInvalid && attn(&s, 8, at(6) + codes - 16) == kInvalid);
  EXPECT(attn(&s, 8, at(7) + codes / 16 - 16) == kInvalid);
  for (int out = 2; out < 6; ++out)
    for (int other = 0; other < 7; ++other)
      if (other != out) EXPECT(write(&s, out, at(other)) == kInvalid);
  for (int out = 0; out < 2; ++out)
    for (int other = 0; other < 7; ++other)
      if (other != out) EXPECT(read(&s, out, at(other)) == kInvalid);
  for (int out = 5; out < 12; ++out)
    for (int other = 0; other < 12; ++other)
      if (other != out) EXPECT(fork(&s, out, at(other)) == kInvalid);
  EXPECT(fork(&s, 8, at(7) + 20) == kInvalid);   // pairs are 8 bytes a row
  for (int out = 4; out < 9; ++out)
    for (int other = 0; other < 9; ++other)
      if (other != out) EXPECT(release(&s, out, at(other)) == kInvalid);
  for (int out = 5; out < 13; ++out)
    for (int other = 0; other < 13; ++other)
      if (other != out) EXPECT(compact(&s, out, at(other)) == kInvalid);

  // the copy
  int64_t sizes[65];
  void* arrays[65];
  for (int i = 0; i < 65; ++i) arrays[i] = as<void>(at(i + 4)), sizes[i] = 1024;
  const int32_t* const pairs = as<int32_t>(at(0));
  auto copy = [&](int64_t pages, int64_t most, int n) {
    return rglru_page_copy(pages, pairs, most, as<int32_t>(at(1)), n, arrays, sizes, nullptr);
  };
  for (int64_t v : big64) EXPECT(copy(v, 0, 2) == kInvalid && copy(100, v, 2) == kInvalid);
  EXPECT(copy(0, 0, 2) == kInvalid && copy(100, 0, 0) == kInvalid && copy(100, 0, 65) == kInvalid && copy(100, 0, -1) == kInvalid);
  EXPECT(rglru_page_copy(100, nullptr, 3, nullptr, 2, arrays, sizes, nullptr) == kInvalid);
  EXPECT(rglru_page_copy(100, pairs, 0, nullptr, 2, nullptr, sizes, nullptr) == kInvalid);
  EXPECT(rglru_page_copy(100, pairs, 0, nullptr, 2, arrays, nullptr, nullptr) == kInvalid);
  EXPECT(rglru_page_copy(100, as<int32_t>(at(0) + 2), 0, nullptr, 2, arrays, sizes, nullptr) == RGLRU_ERR_MISALIGNED);
  EXPECT(rglru_page_copy(100, pairs, 0, as<int32_t>(at(1) + 2), 2, arrays, sizes, nullptr) == RGLRU_ERR_MISALIGNED);
  for (int64_t v : {int64_t(0), int64_t(8), int64_t(1000), int64_t(-16), int64_t(1) << 31, std::numeric_limits<int64_t>::max()}) {
    sizes[1] = v;
    EXPECT(copy(100, 0, 2) == kInvalid);
  }
  sizes[0] = sizes[1] = int64_t(1) << 30;   // together
  EXPECT(copy(100, 0, 2) == kInvalid);
  sizes[0] = sizes[1] = 1024;
  for (uintptr_t v : {uintptr_t(0), at(5) + 8, at(4), at(4) + 100 * 1024 - 16, at(0)}) {
    arrays[1] = as<void>(v);
    EXPECT(rglru_page_copy(100, pairs, 5, nullptr, 2, arrays, sizes, nullptr) == (v == at(5) + 8 ? RGLRU_ERR_MISALIGNED : kInvalid));
  }
  arrays[1] = as<void>(at(5));

  // nothing to do is not an error
  EXPECT(copy(100, 0, 64) == RGLRU_OK && rglru_page_copy(100, nullptr, 0, nullptr, 1, arrays, sizes, nullptr) == RGLRU_OK);
  s = shape();
  s.n_tokens = 0;
  EXPECT(rglru_paged_attn_q4_fwd(&s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                 0, nullptr) == RGLRU_OK);
  EXPECT(rglru_paged_kv_write_q4(&s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr) == RGLRU_OK);
  EXPECT(rglru_paged_kv_read_q4(&s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr) == RGLRU_OK);

  if (g_fail == 0) std::printf("all passed\n");
  return g_fail == 0 ? 0 : 1;
}
