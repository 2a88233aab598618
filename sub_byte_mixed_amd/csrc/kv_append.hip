// Writing and reading a 4-bit key/value cache, gfx950.
//
// Append: rotation of queries and keys (a' = a c - b s, b' = b c + a s over the
// pairs of a head's first dimensions, fp32, not contracted), then keys and
// values as E2M1 with a scale a block, s = RNE(max|x| / 6) and round(x / s) for
// NVFP4, s = 2^(floor(log2 max|x|) - 2) for MXFP4.
//
// Bound by the bytes of the inputs, or, for one token, by latency. A lane has 8
// dimensions of a head's lower half (of the rotated part, then of the rest) and
// the 8 that they pair with, so that a pair is rotated in its registers, an
// access is 16 bytes of input, and a block's maximum is that of 2 (NVFP4) or 4
// (MXFP4) neighbouring lanes. A wave has heads of one token: sequence, page and
// angles are found once a wave.
#include "kv_common.h"

namespace snip {

namespace {

constexpr int kWaves = 4;
// Waves a launch holds at most; more walk on. A grid has fewer than 2^32 threads.
constexpr int64_t kMaxWG = 1 << 20;

__device__ __forceinline__ void load8(const float* p, int64_t off, float (&x)[8]) {
  Raw<true> r;
  load_whole(p, off, r);
  raw_to_f32(r, x);
}

// The 8 elements' share of a block: codes in *w, scale byte in *sc (the same in
// each lane of the block).
template <int FMT>
__device__ __forceinline__ void encode8(float (&x)[8], int e, uint32_t* w, uint32_t* sc) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool finite = fabsf(x[i]) < __builtin_inff();
    if constexpr (FMT == SNIP_NVFP4) x[i] = ldexpf(x[i], -e);   // may leave fp32: the block's scale is the largest then
    m = fmaxf(m, finite ? fabsf(x[i]) : 0.0f);
  }
  float inv;
  if constexpr (FMT == SNIP_NVFP4) {
    m = group_max<2>(m);
    *sc = e4m3_rne(m / 6.0f);
    inv = *sc ? 1.0f / e4m3_val(*sc) : 0.0f;
  } else {
    m = group_max<4>(m);
    const int b = (int)(__float_as_uint(m) >> 23) - 129;   // floor(log2 m) - 2
    const int X = b < -127 ? -127 : b;
    *sc = (uint32_t)(X + 127);
    inv = m > 0.0f ? exp2i(-X) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = __builtin_amdgcn_fmed3f(x[i], -3.0e38f, 3.0e38f) * inv;   // no inf * 0
    x[i] = x[i] != x[i] ? 0.0f : __builtin_amdgcn_fmed3f(r, -8.0f, 8.0f);    // 6 is the largest code
  }
  *w = fp4x8_rne(x);
}

template <int FMT, int D, bool F32>
__global__ __launch_bounds__(64 * kWaves) void kv_append_kernel(KvAppend A) {
  using At = KvAt<FMT, D>;
  constexpr int LPH = D / 16, HPW = 64 / LPH;              // lanes of a head, heads of a wave
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nq = A.q ? A.q_heads : 0, nk = A.k ? A.c.heads : 0;
  const int units = (nq + 2 * nk + HPW - 1) / HPW;         // waves of a token
  const int64_t all = A.tokens * units;
  const int c = lane % LPH;
  const bool turned = 16 * c < A.rot;                      // the part of the head that this lane has
  const int part = turned ? 0 : A.rot, half = ((turned ? A.rot : D) - part) / 2;
  const int lo = part + 8 * (c - part / 16), hi = lo + half;
  int ek = 0, ev = 0;
  if constexpr (FMT == SNIP_NVFP4) {
    if (nk) {
      ek = A.c.texp[0];
      ev = A.c.texp[1];
    }
  }
  for (int64_t u = (int64_t)blockIdx.x * kWaves + wave; u < all; u += (int64_t)gridDim.x * kWaves) {
    const int64_t t = u / units;
    const int h = (int)(u - t * units) * HPW + lane / LPH;
    const int kind = h < nq ? 0 : h < nq + nk ? 1 : h < nq + 2 * nk ? 2 : 3;
    const int hh = kind == 0 ? h : kind == 1 ? h - nq : h - nq - nk;
    // the elements are asked for before the row's place is looked up
    Raw<F32> rx = {}, ry = {};
    if (kind < 3) {
      const void* p = kind == 0 ? A.q : kind == 1 ? A.k : A.v;
      const int64_t off = t * (kind == 0 ? A.ldq : kind == 1 ? A.ldk : A.ldv) + hh * D;
      load_whole(p, off + lo, rx);
      load_whole(p, off + hi, ry);
    }
    const KvRow row = kv_row(A.b, t);
    if (row.seq < 0) continue;
    const int page = nk ? kv_page(A.c, A.b, row.seq, row.pos) : -1;
    float x[8], y[8];
    if (turned && kind < 2) {
      int64_t at = A.pos ? (int64_t)entries(A.pos)[t] : row.pos;
      at = at < 0 ? 0 : at >= A.angles ? A.angles - 1 : at;
      const int64_t o = at * (A.rot / 2);
      if (A.interleaved) {
        float4 cl = *reinterpret_cast<const float4*>(A.cos + o + lo / 2), sl = *reinterpret_cast<const float4*>(A.sin + o + lo / 2);
        float4 ch = *reinterpret_cast<const float4*>(A.cos + o + hi / 2), sh = *reinterpret_cast<const float4*>(A.sin + o + hi / 2);
        const float cc[8] = {cl.x, cl.y, cl.z, cl.w, ch.x, ch.y, ch.z, ch.w};
        const float ss[8] = {sl.x, sl.y, sl.z, sl.w, sh.x, sh.y, sh.z, sh.w};
        raw_to_f32(rx, x);
        raw_to_f32(ry, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[2 * i], b = x[2 * i + 1], p = y[2 * i], q = y[2 * i + 1];
          x[2 * i] = a * cc[i] - b * ss[i];
          x[2 * i + 1] = b * cc[i] + a * ss[i];
          y[2 * i] = p * cc[4 + i] - q * ss[4 + i];
          y[2 * i + 1] = q * cc[4 + i] + p * ss[4 + i];
        }
      } else {
        float cc[8], ss[8];
        load8(A.cos, o + lo, cc);
        load8(A.sin, o + lo, ss);
        raw_to_f32(rx, x);
        raw_to_f32(ry, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = x[i], b = y[i];
          x[i] = a * cc[i] - b * ss[i];
          y[i] = b * cc[i] + a * ss[i];
        }
      }
    } else {
      raw_to_f32(rx, x);
      raw_to_f32(ry, y);
    }
    if (kind == 0) {
      store_whole(A.q_out, false, t * A.ldqo + hh * D + lo, x);
      store_whole(A.q_out, false, t * A.ldqo + hh * D + hi, y);
    }
    if (page < 0) continue;
    // every lane takes part in its block's maximum
    uint32_t wx, wy, sx, sy;
    const int e = kind == 2 ? ev : ek;
    encode8<FMT>(x, e, &wx, &sx);
    encode8<FMT>(y, e, &wy, &sy);
    if (kind != 1 && kind != 2) continue;
    const int at = (int)(row.pos & ((1 << A.c.shift) - 1));
    const bool first = lo % At::BLK == 0;                  // of its block's lanes
    if (kind == 1) {
      const int64_t g = kv_slot(A.c, page, hh, at & ~15);
      uint8_t* pc = A.c.kc + g * (D / 2);
      *reinterpret_cast<uint32_t*>(pc + At::k_code(at, lo)) = wx;
      *reinterpret_cast<uint32_t*>(pc + At::k_code(at, hi)) = wy;
      uint8_t* ps = A.c.ks + g * (D / At::BLK);
      if (first) {
        ps[At::k_scale(at, lo)] = (uint8_t)sx;
        ps[At::k_scale(at, hi)] = (uint8_t)sy;
      }
    } else {
      const int64_t g = kv_slot(A.c, page, hh, at & ~3);
      uint8_t* pc = A.c.vc + g * (D / 2);
      if constexpr (At::V == 4) {
        *reinterpret_cast<uint32_t*>(pc + At::v_code(at, lo)) = wx;
        *reinterpret_cast<uint32_t*>(pc + At::v_code(at, hi)) = wy;
      } else {
        *reinterpret_cast<uint16_t*>(pc + At::v_code(at, lo)) = (uint16_t)wx;
        *reinterpret_cast<uint16_t*>(pc + At::v_code(at, lo + 4)) = (uint16_t)(wx >> 16);
        *reinterpret_cast<uint16_t*>(pc + At::v_code(at, hi)) = (uint16_t)wy;
        *reinterpret_cast<uint16_t*>(pc + At::v_code(at, hi + 4)) = (uint16_t)(wy >> 16);
      }
      uint8_t* ps = A.c.vs + g * (D / At::BLK);
      if (first) {
        ps[At::v_scale(at, lo)] = (uint8_t)sx;
        ps[At::v_scale(at, hi)] = (uint8_t)sy;
      }
    }
  }
}

// Reading back: a lane decodes 8 dimensions of TPW tokens in a row, whose loads
// are in flight together. Bound by the bf16 that it writes, or by latency.
template <int FMT, int D, int TPW>
__global__ __launch_bounds__(64 * kWaves) void kv_gather_kernel(KvGather A) {
  using At = KvAt<FMT, D>;
  constexpr int LPH = D / 8, HPW = 64 / LPH;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nk = A.k ? A.c.heads : 0, nv = A.v ? A.c.heads : 0;
  const int units = (nk + nv + HPW - 1) / HPW;
  const int64_t all = (A.tokens + TPW - 1) / TPW * units;
  const int d = 8 * (lane % LPH);
  const int ek = FMT == SNIP_NVFP4 ? entries(A.c.texp)[0] : 0, ev = FMT == SNIP_NVFP4 ? entries(A.c.texp)[1] : 0;
  for (int64_t u = (int64_t)blockIdx.x * kWaves + wave; u < all; u += (int64_t)gridDim.x * kWaves) {
    const int64_t t0 = u / units * TPW;
    const int h = (int)(u % units) * HPW + lane / LPH;
    const bool key = h < nk, some = h < nk + nv;
    const int hh = some ? (key ? h : h - nk) : 0;
    KvRow row = kv_row(A.b, t0);
    uint32_t w[TPW], b[TPW];
    int seq[TPW], page[TPW];
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      if (i) row = t0 + i < A.tokens ? kv_next(A.b, row, t0 + i - 1) : KvRow{-1, -1, t0 + i + 1};
      seq[i] = row.seq;
      page[i] = kv_page(A.c, A.b, row.seq, row.pos);
      const int at = page[i] < 0 ? 0 : (int)(row.pos & ((1 << A.c.shift) - 1));   // not mapped: any page
      const int64_t g = kv_slot(A.c, page[i] < 0 ? 0 : page[i], hh, key ? at & ~15 : at & ~3);
      const uint8_t* pc = (key ? A.c.kc : A.c.vc) + g * (D / 2);
      const uint8_t* ps = (key ? A.c.ks : A.c.vs) + g * (D / At::BLK);
      if (At::V == 4)
        w[i] = *reinterpret_cast<const uint32_t*>(pc + (key ? At::k_code(at, d) : At::v_code(at, d)));
      else
        w[i] = *reinterpret_cast<const uint16_t*>(pc + (key ? At::k_code(at, d) : At::v_code(at, d))) |
               (uint32_t)*reinterpret_cast<const uint16_t*>(pc + (key ? At::k_code(at, d) + 2 : At::v_code(at, d + 4))) << 16;
      b[i] = ps[key ? At::k_scale(at, d) : At::v_scale(at, d)];
    }
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      if (seq[i] < 0 || !some) continue;
      float q[8];
      fp4x8_dec(w[i], q);
      const int e = FMT == SNIP_NVFP4 ? (key ? ek : ev) : (int)b[i] - 127;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (FMT == SNIP_NVFP4)
          q[j] = ldexpf(q[j] * __builtin_amdgcn_cvt_f32_fp8((int)b[i], 0), e);
        else
          q[j] = b[i] == 255u ? __uint_as_float(0x7FC00000u) : ldexpf(q[j], e);
        if (page[i] < 0) q[j] = 0.0f;
      }
      store_whole(key ? A.k : A.v, false, (t0 + i) * (key ? A.ldk : A.ldv) + hh * D + d, q);
    }
  }
}

int64_t grid_of(int64_t tokens, int heads, int heads_per_wave) {
  const int64_t wg = (tokens * ((heads + heads_per_wave - 1) / heads_per_wave) + kWaves - 1) / kWaves;
  return wg < kMaxWG ? wg : kMaxWG;
}

// fn(format, head_dim) of the pair at run time.
template <typename Fn>
hipError_t dispatch(int format, int dim, Fn fn) {
  auto of = [&](auto f) {
    return dim == 64    ? fn(f, std::integral_constant<int, 64>{})
           : dim == 128 ? fn(f, std::integral_constant<int, 128>{})
                        : fn(f, std::integral_constant<int, 256>{});
  };
  return format == SNIP_NVFP4 ? of(std::integral_constant<int, SNIP_NVFP4>{})
                              : of(std::integral_constant<int, SNIP_MXFP4>{});
}

}  // namespace

hipError_t launch_kv_append(int format, int dim, const KvAppend& a, hipStream_t s) {
  return dispatch(format, dim, [&](auto f, auto d) {
    constexpr int D = decltype(d)::value;
    const int heads = (a.q ? a.q_heads : 0) + (a.k ? 2 * a.c.heads : 0);
    const unsigned grid = (unsigned)grid_of(a.tokens, heads, 1024 / D);
    if (a.type == SNIPOP_F32)
      kv_append_kernel<decltype(f)::value, D, true><<<grid, 64 * kWaves, 0, s>>>(a);
    else
      kv_append_kernel<decltype(f)::value, D, false><<<grid, 64 * kWaves, 0, s>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_kv_gather(int format, int dim, const KvGather& a, hipStream_t s) {
  return dispatch(format, dim, [&](auto f, auto d) {
    constexpr int D = decltype(d)::value;
    const int heads = (a.k ? a.c.heads : 0) + (a.v ? a.c.heads : 0);
    const int64_t wg = grid_of(a.tokens, heads, 512 / D);
    if (a.b.cu && wg >= 8192)                              // more waves than are resident, four times over
      kv_gather_kernel<decltype(f)::value, D, 4><<<(unsigned)grid_of((a.tokens + 3) / 4, heads, 512 / D), 64 * kWaves, 0, s>>>(a);
    else
      kv_gather_kernel<decltype(f)::value, D, 1><<<(unsigned)wg, 64 * kWaves, 0, s>>>(a);
    return hipGetLastError();
  });
}

}  // namespace snip
