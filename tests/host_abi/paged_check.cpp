// Host-side checks of the paged-cache entry points, built with
// AddressSanitizer and UndefinedBehaviorSanitizer around the library's host
// code (host-only compile: no kernel runs): the size query over ordinary and extreme
// shapes, and every refusal, which must come before anything is launched.
// Prints one line per failed expectation and exits nonzero if any failed.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "paged_attn.h"

static int g_fail = 0;

#define EXPECT(cond)                                                   \
  do {                                                                 \
    if (!(cond)) {                                                     \
      std::printf("FAIL line %d: %s\n", __LINE__, #cond);              \
      ++g_fail;                                                        \
    }                                                                  \
  } while (0)

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
static T* fake(uintptr_t at = 0x100000) {  // never dereferenced: every call here is refused
  return reinterpret_cast<T*>(at);
}

static rglru_status_t attn(const rglru_paged_shape_t* s, uintptr_t q = 0x100000, uintptr_t ws = 0x100000, size_t bytes = 0) {
  return rglru_paged_attn_fwd(s, fake<int32_t>(), fake<int32_t>(), fake<int32_t>(), fake<void>(q), fake<void>(), fake<void>(),
                              fake<void>(), fake<float>(), fake<void>(ws), bytes, nullptr);
}
static rglru_status_t plan(const rglru_paged_shape_t* s, int32_t* count_out = fake<int32_t>(0x200000),
                           const int32_t* ctx = fake<int32_t>()) {
  return rglru_page_plan(s, ctx, nullptr, fake<int32_t>(), fake<int32_t>(), fake<int32_t>(), fake<int32_t>(), count_out,
                         fake<int32_t>(), fake<int32_t>(), fake<int32_t>(), fake<int32_t>(), fake<int32_t>(), nullptr);
}
static rglru_status_t write(const rglru_paged_shape_t* s, uintptr_t k = 0x100000) {
  return rglru_paged_kv_write(s, fake<void>(k), fake<void>(), fake<void>(), fake<void>(), fake<int32_t>(), nullptr);
}

int main() {
  const int64_t big64[] = {-1, std::numeric_limits<int64_t>::min(), std::numeric_limits<int64_t>::max(), int64_t(1) << 31,
                           int64_t(1) << 40};
  const int32_t big32[] = {-1, std::numeric_limits<int32_t>::min(), std::numeric_limits<int32_t>::max()};
  rglru_paged_shape_t s = shape();
  EXPECT(rglru_paged_attn_workspace_bytes(nullptr) == 0);
  EXPECT(attn(nullptr) == RGLRU_ERR_INVALID_ARGUMENT && plan(nullptr) == RGLRU_ERR_INVALID_ARGUMENT &&
         write(nullptr) == RGLRU_ERR_INVALID_ARGUMENT);

  // sizes: nonzero, larger batches never need less, a multiple of 256
  for (int io : {0, 1})
    for (int d : {64, 128, 256})
      for (int group : {1, 5, 16, 300})
        for (int64_t t : {int64_t(0), int64_t(1), int64_t(7), int64_t(5000), int64_t(1) << 21}) {
          s = shape();
          s.io_dtype = io;
          s.head_dim = d;
          s.q_heads = s.kv_heads * group;
          s.n_tokens = t;
          const size_t a = rglru_paged_attn_workspace_bytes(&s);
          EXPECT(a > 0 && a % 256 == 0 && a < (size_t(1) << 32));
          s.max_new = 1;
          EXPECT(rglru_paged_attn_workspace_bytes(&s) <= a || t * group <= 32);
        }
  s = shape();
  s.n_pages = (int64_t(1) << 31) / 8 - 1;
  s.page_size = 8;
  s.max_pages = ((int64_t(1) << 31) - (1 << 16)) / 8;
  s.n_seqs = 1 << 16;
  s.q_heads = s.kv_heads = 1;
  s.n_tokens = (int64_t(1) << 31) - (1 << 16);
  EXPECT(rglru_paged_attn_workspace_bytes(&s) > 0);
  s.n_tokens += 1;
  EXPECT(rglru_paged_attn_workspace_bytes(&s) == 0);

  // every refused shape
  auto bad = [](auto change, bool attn_reads, bool plan_reads, bool write_reads) {
    rglru_paged_shape_t b = shape();
    change(b);
    if (attn_reads) EXPECT(attn(&b) == RGLRU_ERR_INVALID_ARGUMENT && rglru_paged_attn_workspace_bytes(&b) == 0);
    if (plan_reads) EXPECT(plan(&b) == RGLRU_ERR_INVALID_ARGUMENT);
    if (write_reads) EXPECT(write(&b) == RGLRU_ERR_INVALID_ARGUMENT);
  };
  for (int64_t v : big64) {
    bad([v](rglru_paged_shape_t& b) { b.n_tokens = v; }, true, true, true);
    bad([v](rglru_paged_shape_t& b) { b.n_pages = v; }, true, true, true);
    if (v != (int64_t(1) << 31) - 1) bad([v](rglru_paged_shape_t& b) { b.q_stride = v < 0 ? v : int64_t(1) << 40; }, true, false, false);
    bad([v](rglru_paged_shape_t& b) { b.kv_stride = v < 0 ? v : int64_t(1) << 40; }, false, false, true);
  }
  for (int32_t v : big32) {
    bad([v](rglru_paged_shape_t& b) { b.n_seqs = v; }, true, true, false);
    bad([v](rglru_paged_shape_t& b) { b.max_pages = v; }, true, true, false);
    bad([v](rglru_paged_shape_t& b) { b.page_size = v; }, true, true, true);
    bad([v](rglru_paged_shape_t& b) { b.q_heads = v; }, true, false, false);
    bad([v](rglru_paged_shape_t& b) { b.kv_heads = v; }, true, false, true);
    bad([v](rglru_paged_shape_t& b) { b.head_dim = v; }, true, false, true);
    bad([v](rglru_paged_shape_t& b) { b.io_dtype = v; }, true, false, true);
    if (v < 0) {
      bad([v](rglru_paged_shape_t& b) { b.max_new = v; }, true, true, false);
      bad([v](rglru_paged_shape_t& b) { b.window = v; }, true, false, false);
    }
  }
  bad([](rglru_paged_shape_t& b) { b.n_pages = 0; }, true, true, true);
  bad([](rglru_paged_shape_t& b) { b.n_seqs = 0; }, true, true, false);
  bad([](rglru_paged_shape_t& b) { b.n_seqs = (1 << 16) + 1; }, true, true, false);
  bad([](rglru_paged_shape_t& b) { b.max_pages = 0; }, true, true, false);
  for (int p : {0, 1, 4, 7, 12, 2048}) bad([p](rglru_paged_shape_t& b) { b.page_size = p; }, true, true, true);
  bad([](rglru_paged_shape_t& b) { b.q_heads = 7; }, true, false, false);
  bad([](rglru_paged_shape_t& b) { b.q_heads = 1; }, true, false, false);
  bad([](rglru_paged_shape_t& b) { b.head_dim = 0; }, true, false, true);
  bad([](rglru_paged_shape_t& b) { b.scale = std::numeric_limits<float>::quiet_NaN(); }, true, false, false);
  bad([](rglru_paged_shape_t& b) { b.scale = std::numeric_limits<float>::infinity(); }, true, false, false);
  bad([](rglru_paged_shape_t& b) { b.q_stride = 8 * 128 - 8; }, true, false, false);
  bad([](rglru_paged_shape_t& b) { b.kv_stride = 2 * 128 - 8; }, false, false, true);

  // unsupported, misaligned, too small, null
  s = shape();
  s.head_dim = 96;
  EXPECT(attn(&s) == RGLRU_ERR_UNSUPPORTED && rglru_paged_attn_workspace_bytes(&s) == 0);
  s.head_dim = 4;
  EXPECT(write(&s) == RGLRU_ERR_UNSUPPORTED);
  s = shape();
  s.q_stride = 8 * 128 + 4;
  EXPECT(attn(&s) == RGLRU_ERR_MISALIGNED);
  s = shape();
  s.kv_stride = 2 * 128 + 4;
  EXPECT(write(&s) == RGLRU_ERR_MISALIGNED);
  s = shape();
  EXPECT(attn(&s, 0x100008) == RGLRU_ERR_MISALIGNED && attn(&s, 0x100000, 0x100080) == RGLRU_ERR_MISALIGNED);
  EXPECT(write(&s, 0x100008) == RGLRU_ERR_MISALIGNED);
  EXPECT(attn(&s, 0x100000, 0x100000, rglru_paged_attn_workspace_bytes(&s) - 1) == RGLRU_ERR_WORKSPACE_TOO_SMALL);
  EXPECT(attn(&s, 0) == RGLRU_ERR_INVALID_ARGUMENT && attn(&s, 0x100000, 0) == RGLRU_ERR_INVALID_ARGUMENT);
  EXPECT(write(&s, 0) == RGLRU_ERR_INVALID_ARGUMENT);
  EXPECT(plan(&s, fake<int32_t>()) == RGLRU_ERR_INVALID_ARGUMENT);   // the old and the new count in one place
  EXPECT(plan(&s, nullptr) == RGLRU_ERR_INVALID_ARGUMENT && plan(&s, fake<int32_t>(0x200000), nullptr) == RGLRU_ERR_INVALID_ARGUMENT);
  EXPECT(plan(&s, fake<int32_t>(0x200002)) == RGLRU_ERR_MISALIGNED);

  // outputs that overlap an input or each other, by a whole array or by its last bytes; every array has a place of its own otherwise
  s = shape();
  {
    const size_t need = rglru_paged_attn_workspace_bytes(&s);
    const int64_t o_size = s.n_tokens * s.q_heads * s.head_dim * 2, cache = s.n_pages * s.page_size * s.kv_heads * s.head_dim * 2;
    auto at = [](int i) { return (uintptr_t(i) + 1) << 32; };
    auto run = [&](int moved, uintptr_t to) {
      uintptr_t p[9];
      for (int i = 0; i < 9; ++i) p[i] = i == moved ? to : at(i);
      return rglru_paged_attn_fwd(&s, fake<int32_t>(p[0]), fake<int32_t>(p[1]), fake<int32_t>(p[2]), fake<void>(p[3]), fake<void>(p[4]),
                                  fake<void>(p[5]), fake<void>(p[6]), fake<float>(p[7]), fake<void>(p[8]), need, nullptr);
    };
    for (int in = 0; in < 6; ++in)
      for (int out = 6; out < 9; ++out) EXPECT(run(out, at(in)) == RGLRU_ERR_INVALID_ARGUMENT);
    EXPECT(run(7, at(6)) == RGLRU_ERR_INVALID_ARGUMENT && run(8, at(7)) == RGLRU_ERR_INVALID_ARGUMENT);
    EXPECT(run(3, at(6) + o_size - 16) == RGLRU_ERR_INVALID_ARGUMENT && run(6, at(5) + cache - 16) == RGLRU_ERR_INVALID_ARGUMENT);
    EXPECT(run(4, at(6) + 16 - cache) == RGLRU_ERR_INVALID_ARGUMENT);
    auto put = [&](int moved, uintptr_t to) {
      uintptr_t p[5];
      for (int i = 0; i < 5; ++i) p[i] = i == moved ? to : at(i);
      return rglru_paged_kv_write(&s, fake<void>(p[0]), fake<void>(p[1]), fake<void>(p[2]), fake<void>(p[3]), fake<int32_t>(p[4]), nullptr);
    };
    EXPECT(put(3, at(2)) == RGLRU_ERR_INVALID_ARGUMENT && put(3, at(2) + cache - 16) == RGLRU_ERR_INVALID_ARGUMENT);
    for (int in : {0, 1, 4}) EXPECT(put(2, at(in)) == RGLRU_ERR_INVALID_ARGUMENT && put(in, at(3) + 16) == RGLRU_ERR_INVALID_ARGUMENT);
    s.n_tokens = (int64_t(1) << 31) - 1;   // the longest span there is
    s.kv_stride = (int64_t(1) << 31) - 8;
    s.kv_heads = 1;
    s.head_dim = 16;
    s.io_dtype = RGLRU_IO_F32;
    EXPECT(put(2, at(0)) == RGLRU_ERR_INVALID_ARGUMENT);
    s = shape();
    auto lay = [&](int moved, uintptr_t to) {
      uintptr_t p[12];
      for (int i = 0; i < 12; ++i) p[i] = i == moved ? to : at(i);
      return rglru_page_plan(&s, fake<int32_t>(p[0]), fake<int32_t>(p[1]), fake<int32_t>(p[2]), fake<int32_t>(p[4]), fake<int32_t>(p[5]),
                             fake<int32_t>(p[3]), fake<int32_t>(p[6]), fake<int32_t>(p[7]), fake<int32_t>(p[8]), fake<int32_t>(p[9]),
                             fake<int32_t>(p[10]), fake<int32_t>(p[11]), nullptr);
    };
    for (int out = 4; out < 12; ++out)
      for (int other = 0; other < 12; ++other)
        if (other != out) EXPECT(lay(out, at(other)) == RGLRU_ERR_INVALID_ARGUMENT);
    EXPECT(lay(9, at(0) + 8) == RGLRU_ERR_INVALID_ARGUMENT && lay(9, at(2) + 12) == RGLRU_ERR_INVALID_ARGUMENT);
  }

  // nothing to do is not an error, and needs no pointers
  s = shape();
  s.n_tokens = 0;
  EXPECT(rglru_paged_attn_fwd(&s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr) ==
         RGLRU_OK);
  EXPECT(rglru_paged_kv_write(&s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr) == RGLRU_OK);

  if (g_fail == 0) std::printf("all passed\n");
  return g_fail == 0 ? 0 : 1;
}
