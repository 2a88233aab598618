// Host-sanitizer (AddressSanitizer + UndefinedBehaviorSanitizer) check of the
// argument validation and sizing of include/snip_kv.h: every entry point is
// called with rejected arguments and the sizing helper over a sweep of shapes.
// None of these calls reaches the GPU. Built like abi_asan_check.cpp; exit
// status 0 iff every status code is the documented one.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/snip_kv.h"

static int g_fail = 0;
#define EXPECT(call, code)                                                                 \
  do {                                                                                     \
    const int rc_ = (call);                                                                \
    if (rc_ != (code)) {                                                                   \
      std::printf("FAIL line %d: %s returned %d, expected %d (%s)\n", __LINE__, #call, rc_, \
                  (code), snip_last_error());                                             \
      ++g_fail;                                                                            \
    } else if (std::strlen(snip_last_error()) == 0) {                                      \
      std::printf("FAIL line %d: %s: no error message\n", __LINE__, #call);                \
      ++g_fail;                                                                            \
    }                                                                                      \
  } while (0)

int main() {
  // fake, 256-aligned device addresses: never dereferenced by rejected calls
  void* const P = reinterpret_cast<void*>(uintptr_t(0x7F0000000000ull));
  void* const Pm = reinterpret_cast<void*>(uintptr_t(0x7F0000000002ull));   // misaligned
  const float* const F = static_cast<const float*>(P);
  const float* const Fm = static_cast<const float*>(Pm);
  const int32_t* const I = static_cast<const int32_t*>(P);
  const int32_t* const Im = static_cast<const int32_t*>(Pm);
  const size_t BIG = size_t(1) << 40;

  // ---- sizing
  const int64_t dims[] = {INT64_MIN, -1, 0, 1, 2, 7, 8, 63, 64, 96, 128, 256, 512, 1024, 1025, 4096, int64_t(1) << 20,
                          (int64_t(1) << 20) + 1, int64_t(1) << 31, int64_t(1) << 40, INT64_MAX};
  size_t sized = 0;
  for (int64_t t : dims)
    for (int64_t s : dims)
      for (int64_t q : dims)
        for (int64_t k : dims)
          for (int64_t d : {int64_t(64), int64_t(128), int64_t(256), int64_t(96), INT64_MIN, INT64_MAX})
            sized += snipkv_attn_workspace(t, s, q, k, d) != 0;

  const snipkv_cache good{SNIP_NVFP4, 64, 4, 128, 10, P, P, P, P, I};
  const snipkv_batch rows{I, 8, 8, I, I, 3};
  auto append = [&](const void* q, const void* k, int type, int64_t tokens, int64_t ld, const float* c, int64_t angles, int64_t rot,
                    const int32_t* pos, const snipkv_cache* cache, const snipkv_batch* batch, void* out) {
    return snipkv_append(q, ld, 8, k, ld, k, ld, type, tokens, c, c, angles, rot, 0, pos, cache, batch, out, ld, nullptr);
  };
  auto attn = [&](const void* q, int64_t heads, int64_t tokens, int64_t ld, float scale, int64_t window, const snipkv_cache* cache,
                  const snipkv_batch* batch, void* out, void* ws, size_t n) {
    return snipkv_attn(q, ld, heads, tokens, cache, batch, scale, window, out, ld, nullptr, ws, n, nullptr);
  };
  auto gather = [&](const snipkv_cache* cache, const snipkv_batch* batch, int64_t tokens, void* k, int64_t ld) {
    return snipkv_gather(cache, batch, tokens, k, ld, nullptr, 0, nullptr);
  };

  // ---- caches
  const int big = INT32_MAX, low = INT32_MIN;
  for (snipkv_cache c : {snipkv_cache{SNIP_NVFP4, 63, 4, 128, 10, P, P, P, P, I}, {SNIP_NVFP4, big, 4, 128, 10, P, P, P, P, I},
                         {SNIP_NVFP4, low, 4, 128, 10, P, P, P, P, I}, {SNIP_NVFP4, 64, big, 128, 10, P, P, P, P, I},
                         {SNIP_NVFP4, 64, low, 128, 10, P, P, P, P, I}, {SNIP_NVFP4, 64, 4, big, 10, P, P, P, P, I},
                         {SNIP_NVFP4, 64, 4, 128, INT64_MAX, P, P, P, P, I}, {SNIP_NVFP4, 64, 4, 128, INT64_MIN, P, P, P, P, I}}) {
    EXPECT(append(P, P, 0, 5, 1024, F, 9, 64, nullptr, &c, &rows, P), SNIP_E_SHAPE);
    EXPECT(attn(P, 8, 5, 1024, 1.0f, 0, &c, &rows, P, P, BIG), SNIP_E_SHAPE);
    EXPECT(gather(&c, &rows, 5, P, 512), SNIP_E_SHAPE);
  }
  for (int f : {low, -1, 0, 1, 4, 7, 8, big}) {
    snipkv_cache c = good;
    c.format = f;
    EXPECT(attn(P, 8, 5, 1024, 1.0f, 0, &c, &rows, P, P, BIG), SNIP_E_FORMAT);
  }
  snipkv_cache c = good;
  c.v_scales = nullptr;
  EXPECT(gather(&c, &rows, 5, P, 512), SNIP_E_NULL);
  c = good;
  c.texp = nullptr;
  EXPECT(gather(&c, &rows, 5, P, 512), SNIP_E_NULL);
  c = good;
  c.k_scales = Pm;
  EXPECT(gather(&c, &rows, 5, P, 512), SNIP_E_ALIGN);
  EXPECT(gather(nullptr, &rows, 5, P, 512), SNIP_E_NULL);

  // ---- batches
  for (snipkv_batch b : {snipkv_batch{I, 8, 0, I, I, 3}, {I, 8, INT64_MAX, I, I, 3}, {I, INT64_MAX, 8, I, I, 3}, {I, 8, INT64_MIN, I, I, 3},
                         {I, 8, 8, I, I, 0}, {I, 8, 8, I, I, INT64_MAX}, {I, 8, 8, I, I, INT64_MIN}, {I, 7, 8, I, I, 3}, {I, 8, 8, I, nullptr, 3}}) {
    EXPECT(append(P, P, 0, 5, 1024, F, 9, 64, nullptr, &good, &b, P), SNIP_E_SHAPE);
    EXPECT(attn(P, 8, 5, 1024, 1.0f, 0, &good, &b, P, P, BIG), SNIP_E_SHAPE);
    EXPECT(gather(&good, &b, 5, P, 512), SNIP_E_SHAPE);
  }
  snipkv_batch b = rows;
  b.table = nullptr;
  EXPECT(gather(&good, &b, 5, P, 512), SNIP_E_NULL);
  b = rows;
  b.lens = Im;
  EXPECT(gather(&good, &b, 5, P, 512), SNIP_E_ALIGN);
  EXPECT(gather(&good, nullptr, 5, P, 512), SNIP_E_NULL);

  // ---- append
  EXPECT(append(nullptr, nullptr, 0, 5, 1024, F, 9, 64, nullptr, &good, &rows, nullptr), SNIP_E_NULL);
  EXPECT(append(P, P, 0, 5, 1024, F, 9, 64, nullptr, &good, &rows, nullptr), SNIP_E_NULL);
  EXPECT(append(P, P, 7, 5, 1024, F, 9, 64, nullptr, &good, &rows, P), SNIP_E_FORMAT);
  for (int64_t t : {INT64_MIN, int64_t(0), INT64_MAX})
    EXPECT(append(P, P, 0, t, 1024, F, 9, 64, nullptr, &good, &rows, P), SNIP_E_SHAPE);
  for (int64_t ld : {INT64_MIN, int64_t(0), int64_t(1023), INT64_MAX, INT64_MAX - 7})
    EXPECT(append(P, P, 0, 5, ld, F, 9, 64, nullptr, &good, &rows, P), SNIP_E_SHAPE);
  for (int64_t r : {INT64_MIN, int64_t(32), int64_t(192), INT64_MAX})
    EXPECT(append(P, P, 0, 5, 1024, F, 9, r, nullptr, &good, &rows, P), SNIP_E_SHAPE);
  for (int64_t n : {INT64_MIN, int64_t(0), INT64_MAX})
    EXPECT(append(P, P, 0, 5, 1024, F, n, 64, nullptr, &good, &rows, P), SNIP_E_SHAPE);
  EXPECT(append(P, P, 0, 5, 1024, nullptr, 9, 64, nullptr, &good, &rows, P), SNIP_E_NULL);
  EXPECT(append(P, P, 0, 5, 1024, Fm, 9, 64, nullptr, &good, &rows, P), SNIP_E_ALIGN);
  EXPECT(append(P, P, 0, 5, 1024, F, 9, 64, Im, &good, &rows, P), SNIP_E_ALIGN);
  EXPECT(append(Pm, P, 0, 5, 1024, F, 9, 64, nullptr, &good, &rows, P), SNIP_E_ALIGN);

  // ---- gather
  EXPECT(snipkv_gather(&good, &rows, 5, nullptr, 0, nullptr, 0, nullptr), SNIP_E_NULL);
  for (int64_t ld : {INT64_MIN, int64_t(511), INT64_MAX}) EXPECT(gather(&good, &rows, 5, P, ld), SNIP_E_SHAPE);
  EXPECT(gather(&good, &rows, 5, Pm, 512), SNIP_E_ALIGN);

  // ---- attention
  EXPECT(attn(nullptr, 8, 5, 1024, 1.0f, 0, &good, &rows, P, P, BIG), SNIP_E_NULL);
  for (int64_t h : {INT64_MIN, int64_t(0), int64_t(6), INT64_MAX})
    EXPECT(attn(P, h, 5, 1024, 1.0f, 0, &good, &rows, P, P, BIG), SNIP_E_SHAPE);
  for (float s : {0.0f, -1.0f, INFINITY, NAN}) EXPECT(attn(P, 8, 5, 1024, s, 0, &good, &rows, P, P, BIG), SNIP_E_SHAPE);
  for (int64_t w : {INT64_MIN, int64_t(-1)}) EXPECT(attn(P, 8, 5, 1024, 1.0f, w, &good, &rows, P, P, BIG), SNIP_E_SHAPE);
  EXPECT(attn(P, 8, 5, 1024, 1.0f, 0, &good, &rows, Pm, P, BIG), SNIP_E_ALIGN);
  EXPECT(attn(P, 8, 5, 1024, 1.0f, 0, &good, &rows, P, Pm, BIG), SNIP_E_ALIGN);
  EXPECT(attn(P, 8, 5, 1024, 1.0f, 0, &good, &rows, P, nullptr, BIG), SNIP_E_WORKSPACE);
  EXPECT(attn(P, 8, 5, 1024, 1.0f, 0, &good, &rows, P, P, 16), SNIP_E_WORKSPACE);

  std::printf("{\"failures\": %d, \"sized\": %zu}\n", g_fail, sized);
  return g_fail ? 1 : 0;
}
