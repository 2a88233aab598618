// Host-sanitizer (AddressSanitizer + UndefinedBehaviorSanitizer) check of the
// argument validation and sizing of include/snip_ops.h: every entry point is
// called with rejected arguments and every sizing helper over a sweep of shapes.
// None of these calls reaches the GPU. Built like abi_asan_check.cpp; exit
// status 0 iff every status code is the documented one.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/snip_ops.h"

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
  void* const P2 = reinterpret_cast<void*>(uintptr_t(0x7F0000100000ull));
  void* const Pm = reinterpret_cast<void*>(uintptr_t(0x7F0000000002ull));   // misaligned
  float* const F = static_cast<float*>(P);
  float* const Fm = static_cast<float*>(Pm);
  snip_stats* const ST = static_cast<snip_stats*>(P2);
  int32_t* const E = static_cast<int32_t*>(P2);
  const int B = SNIPOP_BF16, W = SNIPOP_F32;
  const size_t BIG = 1 << 30;

  // ---- sizing
  const int64_t dims[] = {-1, 0, 1, 7, 16, 64, 512, 1000, 1024, 1032, 4096, 8192, 8200, 16384, 16400, 28672,
                          int64_t(1) << 31, int64_t(1) << 40, INT64_MAX};
  size_t acc = 0;
  for (int64_t rows : dims)
    for (int64_t cols : dims) {
      acc += snipop_rmsnorm_bwd_workspace(rows, cols);
      for (int f = -1; f <= 8; ++f)
        acc += snipop_rmsnorm_fwd_workspace(rows, cols, f) + snipop_swiglu_fwd_workspace(rows, cols, f);
    }
  if (snipop_rmsnorm_bwd_workspace(4, SNIPOP_NORM_MAX_COLS + 1) != 0 || snipop_swiglu_fwd_workspace(4, 40, SNIP_FP8_E4M3) != 0)
    ++g_fail;

  snip_qtensor q{SNIP_FP8_E4M3, 0, 4, 64, P, P2, E};
  snip_qtensor qn{SNIP_NVFP4, 0, 4, 64, P, P2, E};
  snip_qtensor qo{SNIP_FP8_E4M3, 0, 8, 64, P, P2, E};
  snip_qtensor qb{SNIP_BF16, 0, 4, 64, P, P2, E};
  snip_qtensor qx{9, 0, 4, 64, P, P2, E};
  snip_qtensor qs{SNIP_NVFP4, 0, 4, 64, P, nullptr, E};

  // ---- norm forward
  auto norm = [&](const void* x, int xt, int64_t ldx, int64_t rows, int64_t cols, float eps, void* y, const snip_qtensor* out,
                  int rnd, const float* amax, snip_stats* st, size_t n) {
    return snipop_rmsnorm_fwd(x, xt, ldx, P, B, 64, P, B, rows, cols, eps, nullptr, 0, 0, y, B, 64, nullptr, out, rnd, 0, 0,
                              amax, st, n ? P : nullptr, n, nullptr);
  };
  EXPECT(norm(nullptr, B, 64, 4, 64, 1e-5f, P, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_NULL);
  EXPECT(norm(P, B, 64, 4, 64, 1e-5f, nullptr, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_NULL);
  EXPECT(norm(P, B, 64, 4, 64, 1e-5f, P, nullptr, 0, nullptr, ST, BIG), SNIP_E_NULL);
  EXPECT(norm(P, B, 64, 4, 64, 1e-5f, P, &qs, 0, nullptr, nullptr, BIG), SNIP_E_NULL);
  EXPECT(norm(P, B, 64, 0, 64, 1e-5f, P, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_SHAPE);
  EXPECT(norm(P, B, 64, INT64_MAX, 64, 1e-5f, P, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_SHAPE);
  EXPECT(norm(P, B, INT64_MAX, 4, 64, 1e-5f, P, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_SHAPE);
  EXPECT(norm(P, B, int64_t(1) << 40, int64_t(1) << 40, 64, 1e-5f, P, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_SHAPE);
  EXPECT(norm(P, W, 66, 4, 64, 1e-5f, P, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_SHAPE);
  EXPECT(norm(P, B, 64, 4, 64, NAN, P, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_SHAPE);
  EXPECT(norm(P, B, 64, 4, 64, -1.0f, P, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_SHAPE);
  EXPECT(norm(P, B, 64, 4, 64, 1e-5f, P, &qo, 0, nullptr, nullptr, BIG), SNIP_E_SHAPE);
  EXPECT(norm(Pm, B, 64, 4, 64, 1e-5f, P, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_ALIGN);
  EXPECT(norm(P, B, 64, 4, 64, 1e-5f, P, &q, 0, Fm, nullptr, BIG), SNIP_E_ALIGN);
  EXPECT(norm(P, 2, 64, 4, 64, 1e-5f, P, nullptr, 0, nullptr, nullptr, BIG), SNIP_E_FORMAT);
  EXPECT(norm(P, B, 64, 4, 64, 1e-5f, P, &qb, 0, nullptr, nullptr, BIG), SNIP_E_FORMAT);
  EXPECT(norm(P, B, 64, 4, 64, 1e-5f, P, &qx, 0, nullptr, nullptr, BIG), SNIP_E_FORMAT);
  EXPECT(norm(P, B, 64, 4, 64, 1e-5f, P, &q, 3, nullptr, nullptr, BIG), SNIP_E_FORMAT);
  EXPECT(norm(P, B, 64, 4, 64, 1e-5f, P, &q, 0, nullptr, nullptr, 0), SNIP_E_WORKSPACE);
  EXPECT(norm(P, B, 64, 4, 64, 1e-5f, P, &qn, 0, F, ST, 64), SNIP_E_WORKSPACE);

  // ---- norm backward
  auto nbwd = [&](const void* dy, int yt, int64_t ldy, int64_t rows, int64_t cols, void* dx, float* dg, size_t n) {
    return snipop_rmsnorm_bwd(dy, yt, ldy, P, B, 64, P, B, F, nullptr, 0, 0, rows, cols, dx, B, 64, dg, P, n, nullptr);
  };
  EXPECT(nbwd(nullptr, B, 64, 4, 64, P, F, BIG), SNIP_E_NULL);
  EXPECT(nbwd(P, B, 64, 4, 64, nullptr, nullptr, BIG), SNIP_E_NULL);
  EXPECT(nbwd(P, B, 64, -4, 64, P, F, BIG), SNIP_E_SHAPE);
  EXPECT(nbwd(P, B, 64, 4, SNIPOP_NORM_MAX_COLS + 8, P, F, BIG), SNIP_E_SHAPE);
  EXPECT(nbwd(P, B, 63, 4, 64, P, F, BIG), SNIP_E_SHAPE);
  EXPECT(nbwd(P, -1, 64, 4, 64, P, F, BIG), SNIP_E_FORMAT);
  EXPECT(nbwd(Pm, B, 64, 4, 64, P, F, BIG), SNIP_E_ALIGN);
  EXPECT(nbwd(P, B, 64, 4, 64, P, Fm, BIG), SNIP_E_ALIGN);
  EXPECT(nbwd(P, B, 64, 4, 64, P, F, 16), SNIP_E_WORKSPACE);

  // ---- SwiGLU
  auto gate = [&](const void* g, int t, int64_t ldg, int64_t rows, int64_t cols, void* y, const snip_qtensor* out, size_t n) {
    return snipop_swiglu_fwd(g, ldg, P, 64, t, rows, cols, y, B, 64, out, 0, 0, 0, nullptr, nullptr, P, n, nullptr);
  };
  EXPECT(gate(nullptr, B, 64, 4, 64, P, nullptr, BIG), SNIP_E_NULL);
  EXPECT(gate(P, B, 64, 4, 64, nullptr, nullptr, BIG), SNIP_E_NULL);
  EXPECT(gate(P, B, 64, 4, (int64_t(1) << 31) + 1, P, nullptr, BIG), SNIP_E_SHAPE);
  EXPECT(gate(P, B, 60, 4, 64, P, nullptr, BIG), SNIP_E_SHAPE);
  EXPECT(gate(P, 5, 64, 4, 64, P, nullptr, BIG), SNIP_E_FORMAT);
  EXPECT(gate(Pm, B, 64, 4, 64, P, nullptr, BIG), SNIP_E_ALIGN);
  EXPECT(gate(P, B, 64, 4, 64, P, &q, 8), SNIP_E_WORKSPACE);
  auto gbwd = [&](const void* dy, int64_t ldy, int t, int64_t rows, void* dg, void* du) {
    return snipop_swiglu_bwd(dy, t, ldy, P, 64, P, 64, B, rows, 64, dg, 64, du, 64, B, nullptr);
  };
  EXPECT(gbwd(nullptr, 64, B, 4, P, P2), SNIP_E_NULL);
  EXPECT(gbwd(P, 64, B, 4, nullptr, nullptr), SNIP_E_NULL);
  EXPECT(gbwd(P, 64, B, 0, P, P2), SNIP_E_SHAPE);
  EXPECT(gbwd(P, 56, B, 4, P, P2), SNIP_E_SHAPE);
  EXPECT(gbwd(P, 64, 3, 4, P, P2), SNIP_E_FORMAT);
  EXPECT(gbwd(P, 64, B, 4, Pm, P2), SNIP_E_ALIGN);

  // ---- tokens x weights
  auto gemv = [&](const void* x, int64_t ldx, int64_t m, int f, int64_t n, int64_t k, void* y, int yt, int64_t ldy) {
    const snip_qtensor w{f, 0, n, k, P, P2, E};
    return snipop_qgemv(x, ldx, m, &w, y, yt, ldy, nullptr);
  };
  EXPECT(snipop_qgemv(P, 64, 1, nullptr, P, W, 64, nullptr), SNIP_E_NULL);
  EXPECT(gemv(nullptr, 64, 1, SNIP_NVFP4, 8, 64, P, W, 8), SNIP_E_NULL);
  EXPECT(gemv(P, 64, 0, SNIP_NVFP4, 8, 64, P, W, 8), SNIP_E_SHAPE);
  EXPECT(gemv(P, 64, 17, SNIP_NVFP4, 8, 64, P, W, 8), SNIP_E_SHAPE);
  EXPECT(gemv(P, 64, 1, SNIP_NVFP4, 8, 48, P, W, 8), SNIP_E_SHAPE);
  EXPECT(gemv(P, 60, 1, SNIP_NVFP4, 8, 64, P, W, 8), SNIP_E_SHAPE);
  EXPECT(gemv(P, 64, 1, SNIP_NVFP4, 8, 64, P, W, 7), SNIP_E_SHAPE);
  EXPECT(gemv(P, 64, 1, SNIP_NVFP4, INT64_MAX, 64, P, W, INT64_MAX), SNIP_E_SHAPE);
  EXPECT(gemv(P, int64_t(1) << 25, 1, SNIP_MXFP4, int64_t(1) << 31, int64_t(1) << 25, P, W, int64_t(1) << 31), SNIP_E_SHAPE);
  EXPECT(gemv(P, 64, 1, SNIP_BF16, 8, 64, P, W, 8), SNIP_E_FORMAT);
  EXPECT(gemv(P, 64, 1, SNIP_NVFP4, 8, 64, P, 2, 8), SNIP_E_FORMAT);
  EXPECT(gemv(Pm, 64, 1, SNIP_NVFP4, 8, 64, P, W, 8), SNIP_E_ALIGN);
  EXPECT(gemv(P, 64, 1, SNIP_NVFP4, 8, 64, Pm, W, 8), SNIP_E_ALIGN);

  std::printf("{\"failures\": %d, \"sized\": %zu}\n", g_fail, acc);
  return g_fail ? 1 : 0;
}
