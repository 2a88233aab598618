// Host helpers shared by the entry points of snip.h (api.hip) and of
// snip_ops.h (ops_api.hip): the thread's error message, format facts,
// descriptor checks and workspace carving.
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "kernels.h"

namespace snip {

inline std::string& last_error() {
  static thread_local std::string e;
  return e;
}

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  try {
    last_error() = buf;
  } catch (...) {           // no memory for the message: the code still tells
  }
  return code;
}

inline int ok() {
  last_error().clear();
  return SNIP_OK;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
constexpr size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Formats a qtensor may hold (the FP4 design-space variants included) and
// the formats the GEMM and layer calls take.
inline bool valid_format(int f) { return f >= SNIP_BF16 && f <= SNIP_FP4_BF16_B32; }
inline bool gemm_format(int f) { return f >= SNIP_BF16 && f <= SNIP_MXFP4; }
inline bool fp4_variant(int f) { return f >= SNIP_FP4_E4M3_B32 && f <= SNIP_FP4_BF16_B32; }
inline int block_of(int f) {
  return (f == SNIP_MXFP4 || f == SNIP_FP4_E4M3_B32 || f == SNIP_FP4_BF16_B32) ? 32 : 16;
}
inline bool has_scales(int f) { return f == SNIP_NVFP4 || f == SNIP_MXFP4 || fp4_variant(f); }
inline bool has_texp(int f) { return f == SNIP_NVFP4 || f == SNIP_FP8_E4M3 || f == SNIP_FP4_E4M3_B32; }
inline bool needs_amax(int f) { return has_texp(f); }

inline int64_t code_bytes(int f, int64_t rows, int64_t k) {
  if (f == SNIP_NVFP4 || f == SNIP_MXFP4 || fp4_variant(f)) return rows * k / 2;
  if (f == SNIP_FP8_E4M3) return rows * k;
  if (f == SNIP_BF16) return rows * k * 2;
  return -1;
}
inline int64_t scale_bytes(int f, int64_t rows, int64_t k) {
  if (!has_scales(f)) return 0;
  const int per = (f == SNIP_FP4_BF16_B16 || f == SNIP_FP4_BF16_B32) ? 2 : 1;
  return rows * (k / block_of(f)) * per;
}

constexpr size_t kAlign = 256;

// Bump allocator over the caller's workspace.
struct Carver {
  uint8_t* base;
  size_t used = 0;
  explicit Carver(void* p) : base(static_cast<uint8_t*>(p)) {}
  uint8_t* take(size_t n) {
    uint8_t* p = base + used;
    used += align_up(n, kAlign);
    return p;
  }
};

inline int hip_check(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(SNIP_E_HIP, "%s: %s", what, hipGetErrorString(e));
  return SNIP_OK;
}

inline int validate_qtensor(const snip_qtensor* q, const char* name, bool need_codes = true) {
  if (!q) return fail(SNIP_E_NULL, "%s: descriptor is NULL", name);
  if (!valid_format(q->format)) return fail(SNIP_E_FORMAT, "%s: unknown format %d", name, q->format);
  if (q->rows <= 0 || q->k <= 0) return fail(SNIP_E_SHAPE, "%s: rows=%lld k=%lld must be > 0", name,
                                           (long long)q->rows, (long long)q->k);
  if (q->k % block_of(q->format)) return fail(SNIP_E_SHAPE, "%s: k=%lld not a multiple of %d", name,
                                             (long long)q->k, block_of(q->format));
  if (need_codes && !q->codes) return fail(SNIP_E_NULL, "%s: codes is NULL", name);
  if (has_scales(q->format) && !q->scales) return fail(SNIP_E_NULL, "%s: scales is NULL", name);
  if (has_texp(q->format) && !q->tensor_exp) return fail(SNIP_E_NULL, "%s: tensor_exp is NULL", name);
  if (!aligned(q->codes, 16) || !aligned(q->scales, 16) || !aligned(q->tensor_exp, 4))
    return fail(SNIP_E_ALIGN, "%s: device pointers must be 16-byte aligned", name);
  return SNIP_OK;
}

}  // namespace snip
