// Host-sanitizer check of include/snip_kv.h with matrices that are absent: what
// describes them may hold anything. Every call is rejected for another argument
// and none reaches the GPU. Built like abi_asan_check.cpp; exit status 0 iff every
// status code is the documented one.
#include <cstdint>
#include <cstdio>

#include "../../include/snip_kv.h"

int main() {
  // fake, 256-aligned device addresses: never dereferenced by rejected calls
  void* const P = reinterpret_cast<void*>(uintptr_t(0x7F0000000000ull));
  const float* const F = static_cast<const float*>(P);
  const int32_t* const I = static_cast<const int32_t*>(P);
  const snipkv_batch rows{I, 8, 8, I, I, 3};
  const int64_t any[] = {INT64_MIN, -1, 0, 1, 1023, INT64_MAX / 64, INT64_MAX - 7, INT64_MAX};
  int failures = 0, calls = 0;
  auto expect = [&](int rc, const char* what, int64_t v) {
    ++calls;
    if (rc == SNIP_E_SHAPE) return;
    std::printf("FAIL %s %lld: returned %d (%s)\n", what, (long long)v, rc, snip_last_error());
    ++failures;
  };
  for (int dim : {64, 128, 256}) {
    const snipkv_cache cache{SNIP_NVFP4, 64, 4, dim, 10, P, P, P, P, I};
    for (int64_t v : any) {
      // rot_dim = 32 is what is refused
      expect(snipkv_append(nullptr, v, v, P, 1024, P, 1024, SNIPOP_BF16, 5, F, F, 9, 32, 0, nullptr, &cache, &rows, nullptr, v, nullptr),
             "no queries", v);
      expect(snipkv_append(P, 2048, 8, nullptr, v, nullptr, v, SNIPOP_BF16, 5, F, F, 9, 32, 0, nullptr, &cache, &rows, P, 2048, nullptr),
             "no keys", v);
      // a leading dimension of one element is
      expect(snipkv_gather(&cache, &rows, 5, P, 1, nullptr, v, nullptr), "no values", v);
      expect(snipkv_gather(&cache, &rows, 5, nullptr, v, P, 1, nullptr), "no keys out", v);
    }
  }
  std::printf("{\"failures\": %d, \"calls\": %d}\n", failures, calls);
  return failures ? 1 : 0;
}
