// Device helpers shared by the kernels of the 4-bit key/value cache: where a
// row's token lies.
#pragma once

#include "kv.h"
#include "row_common.h"

namespace snip {

// Loads whose address is the same in the wave's lanes, of what the launch does
// not write: scalar, and not waited for in order with the vector loads.
typedef const __attribute__((address_space(4))) int32_t* Entries;
__device__ __forceinline__ Entries entries(const int32_t* p) { return (Entries)(uintptr_t)p; }

// The sequence that holds x, f ascending: the number of b in 0 .. n with
// f(b) <= x, less one; -1 before the first, n behind the last. The wave narrows
// 64 ways a step, so that up to 63 sequences take one load's latency.
template <typename F>
__device__ __forceinline__ int kv_find(int n, int64_t x, F f) {
  const int lane = threadIdx.x & 63;
  int lo = 0, count = n + 1;                           // f(lo - 1) <= x < f(lo + count)
  while (count > 0) {
    const int step = (count + 63) >> 6;
    const int i = lane * step + step - 1;              // the last of this lane's share
    const bool le = i < count && f(lo + i) <= x;
    const int whole = __popcll(__ballot(le));
    lo += whole * step;
    if (step == 1) break;
    count = count - whole * step < step - 1 ? count - whole * step : step - 1;
  }
  return __builtin_amdgcn_readfirstlane(lo) - 1;
}

// fn(format, head_dim) of the pair at run time.
template <typename Fn>
hipError_t kv_dispatch(int format, int dim, Fn fn) {
  auto of = [&](auto f) {
    return dim == 64    ? fn(f, std::integral_constant<int, 64>{})
           : dim == 128 ? fn(f, std::integral_constant<int, 128>{})
                        : fn(f, std::integral_constant<int, 256>{});
  };
  return format == SNIP_NVFP4 ? of(std::integral_constant<int, SNIP_NVFP4>{}) : of(std::integral_constant<int, SNIP_MXFP4>{});
}

struct KvRow {
  int seq;                     // < 0: nobody's
  int64_t pos, end;            // position; the sequence's last row and one
};

// Sequence and position of row t.
__device__ __forceinline__ KvRow kv_row(const KvBatch& b, int64_t t) {
  if (!b.cu) return t < b.seqs ? KvRow{(int)t, (int64_t)entries(b.lens)[t] - 1, t + 1} : KvRow{-1, -1, t + 1};
  const int s = kv_find(b.seqs, t, [&](int i) { return (int64_t)b.cu[i]; });
  if (s < 0 || s >= b.seqs) return KvRow{-1, -1, t + 1};
  const int64_t end = entries(b.cu)[s + 1];
  return KvRow{s, (int64_t)entries(b.lens)[s] - (end - t), end};
}

// Row t + 1, after row t.
__device__ __forceinline__ KvRow kv_next(const KvBatch& b, const KvRow& r, int64_t t) {
  if (r.seq >= 0 && t + 1 < r.end) return KvRow{r.seq, r.pos + 1, r.end};
  return kv_row(b, t + 1);
}

// Number of a page, or -1 where the position is not mapped.
__device__ __forceinline__ int kv_page(const KvCache& c, const KvBatch& b, int seq, int64_t pos) {
  if (seq < 0 || pos < 0 || pos >= b.max_len) return -1;
  const int p = entries(b.table + (int64_t)seq * b.table_ld)[pos >> c.shift];
  return p >= 0 && p < c.pages ? p : -1;
}

// Where head h of token `at` of a page lies, in tokens from the buffers' start.
__device__ __forceinline__ int64_t kv_slot(const KvCache& c, int page, int h, int at) {
  return (((int64_t)page * c.heads + h) << c.shift) + at;
}

// Byte offsets of dimension d of the token `at` (of its page), from the first
// token of its 16 (keys) or 4 (values).
template <int FMT, int D>
struct KvAt {
  static constexpr int BLK = FMT == SNIP_NVFP4 ? 16 : 32;
  static constexpr int P = kv_key_piece(D), S = kv_scale_piece(D, BLK), V = kv_value_piece(D);
  static __device__ __forceinline__ int k_code(int at, int d) { return (d / 2 / P * 16 + at % 16) * P + d / 2 % P; }
  static __device__ __forceinline__ int k_scale(int at, int d) { return (d / BLK / S * 16 + at % 16) * S + d / BLK % S; }
  static __device__ __forceinline__ int v_code(int at, int d) { return (d / 2 / V * 4 + at % 4) * V + d / 2 % V; }
  static __device__ __forceinline__ int v_scale(int at, int d) { return d / BLK * 4 + at % 4; }
};

}  // namespace snip
