// Writing and reading a 4-bit key/value cache, gfx950.
//
// Append: rotation of queries and keys (a' = a c - b s, b' = b c + a s over the
// pairs of a head's first dimensions, fp32, not contracted), then keys and
// values as E2M1 with a scale a block, s = RNE(max|x| / 6) and round(x / s) for
// NVFP4, s = 2^(floor(log2 max|x|) - 2) for MXFP4.
//
// Bound by the bytes of the inputs (8192 tokens of 32 + 2 x 32 heads of 128, fp32:
// 517 MB in 115 us, 4.5 TB/s), or, for one token, by latency (3 us). A lane has 8
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
// Workgroups of single tokens from which a wave takes four: a fourth of the waves
// still fill the GPU (8192 tokens of 96 heads: 169 -> 153 us with the gather; 1840
// tokens of 80 heads gain nothing, 31 and 32).
constexpr int64_t kLong = 8192;

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

// TPW tokens in a row to a wave: one, or four in long calls. Then a workgroup has
// 16 tokens of the same heads, so that what they share -- 16 bytes of values and 4
// of their scales, 256 bytes of keys -- is written by one wave at once, or within
// one cache.
template <int FMT, int D, bool F32, int TPW>
__global__ __launch_bounds__(64 * kWaves) void kv_append_kernel(KvAppend A) {
  using At = KvAt<FMT, D>;
  constexpr int LPH = D / 16, HPW = 64 / LPH;              // lanes of a head, heads of a wave
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nq = A.q ? A.q_heads : 0, nk = A.k ? A.c.heads : 0;
  const int units = (nq + 2 * nk + HPW - 1) / HPW;         // waves of a token
  const int64_t all = TPW == 1 ? A.tokens * units : (A.tokens + TPW * kWaves - 1) / (TPW * kWaves) * units * kWaves;
  const int c = lane % LPH;
  const bool turned = 16 * c < A.rot;                      // the part of the head that this lane has
  const int part = turned ? 0 : A.rot, half = ((turned ? A.rot : D) - part) / 2;
  const int lo = part + 8 * (c - part / 16), hi = lo + half;
  const bool first = lo % At::BLK == 0;                    // of its block's lanes
  int ek = 0, ev = 0;
  if constexpr (FMT == SNIP_NVFP4) {
    if (nk) {
      ek = entries(A.c.texp)[0];
      ev = entries(A.c.texp)[1];
    }
  }
  for (int64_t u = (int64_t)blockIdx.x * kWaves + wave; u < all; u += (int64_t)gridDim.x * kWaves) {
    const int64_t t0 = TPW == 1 ? u / units : (u / kWaves / units * kWaves + wave) * TPW;
    const int h = (int)((TPW == 1 ? u : u / kWaves) % units) * HPW + lane / LPH;
    const int kind = h < nq ? 0 : h < nq + nk ? 1 : h < nq + 2 * nk ? 2 : 3;
    const int hh = kind == 0 ? h : kind == 1 ? h - nq : h - nq - nk;
    // the elements are asked for before the rows' places are looked up
    Raw<F32> rx[TPW], ry[TPW];
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      rx[i] = {};
      ry[i] = {};
      if (kind < 3 && t0 + i < A.tokens) {
        const void* p = kind == 0 ? A.q : kind == 1 ? A.k : A.v;
        const int64_t off = (t0 + i) * (kind == 0 ? A.ldq : kind == 1 ? A.ldk : A.ldv) + hh * D;
        load_whole(p, off + lo, rx[i]);
        load_whole(p, off + hi, ry[i]);
      }
    }
    KvRow row[TPW];
    int page[TPW];
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      row[i] = t0 + i >= A.tokens ? KvRow{-1, -1, t0 + i + 1} : i ? kv_next(A.b, row[i - 1], t0 + i - 1) : kv_row(A.b, t0);
      page[i] = nk ? kv_page(A.c, A.b, row[i].seq, row[i].pos) : -1;
    }
    uint32_t wx[TPW], wy[TPW], sx[TPW], sy[TPW];
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      if (row[i].seq < 0) continue;
      const int64_t t = t0 + i;
      float x[8], y[8];
      raw_to_f32(rx[i], x);
      raw_to_f32(ry[i], y);
      if (turned && kind < 2) {
        int64_t at = A.pos ? (int64_t)entries(A.pos)[t] : row[i].pos;
        at = at < 0 ? 0 : at >= A.angles ? A.angles - 1 : at;
        const int64_t o = at * (A.rot / 2);
        float cc[8], ss[8];
        if (A.interleaved) {                               // 4 angles of the lower elements, 4 of the upper
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float4 c4 = *reinterpret_cast<const float4*>(A.cos + o + (k ? hi : lo) / 2);
            const float4 s4 = *reinterpret_cast<const float4*>(A.sin + o + (k ? hi : lo) / 2);
            cc[4 * k] = c4.x, cc[4 * k + 1] = c4.y, cc[4 * k + 2] = c4.z, cc[4 * k + 3] = c4.w;
            ss[4 * k] = s4.x, ss[4 * k + 1] = s4.y, ss[4 * k + 2] = s4.z, ss[4 * k + 3] = s4.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = x[2 * k], b = x[2 * k + 1], p = y[2 * k], q = y[2 * k + 1];
            x[2 * k] = a * cc[k] - b * ss[k];
            x[2 * k + 1] = b * cc[k] + a * ss[k];
            y[2 * k] = p * cc[4 + k] - q * ss[4 + k];
            y[2 * k + 1] = q * cc[4 + k] + p * ss[4 + k];
          }
        } else {
          load8(A.cos, o + lo, cc);
          load8(A.sin, o + lo, ss);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float a = x[k], b = y[k];
            x[k] = a * cc[k] - b * ss[k];
            y[k] = b * cc[k] + a * ss[k];
          }
        }
      }
      if (kind == 0) {
        store_whole(A.q_out, false, t * A.ldqo + hh * D + lo, x);
        store_whole(A.q_out, false, t * A.ldqo + hh * D + hi, y);
      }
      if (page[i] < 0) continue;
      // every lane takes part in its block's maximum
      const int e = kind == 2 ? ev : ek;
      encode8<FMT>(x, e, &wx[i], &sx[i]);
      encode8<FMT>(y, e, &wy[i], &sy[i]);
      if (kind == 1) {
        const int at = (int)(row[i].pos & ((1 << A.c.shift) - 1));
        const int64_t g = kv_slot(A.c, page[i], hh, at & ~15);
        uint8_t* pc = A.c.kc + g * (D / 2);
        *reinterpret_cast<uint32_t*>(pc + At::k_code(at, lo)) = wx[i];
        *reinterpret_cast<uint32_t*>(pc + At::k_code(at, hi)) = wy[i];
        uint8_t* ps = A.c.ks + g * (D / At::BLK);
        if (first) {
          ps[At::k_scale(at, lo)] = (uint8_t)sx[i];
          ps[At::k_scale(at, hi)] = (uint8_t)sy[i];
        }
      }
    }
    // values: four tokens that share their 16 bytes, or each for itself
    bool four = TPW == 4 && page[0] >= 0 && (row[0].pos & 3) == 0;
#pragma unroll
    for (int i = 1; i < TPW; ++i) four = four && row[i].seq == row[0].seq && page[i] == page[0];
    if (kind != 2) continue;
    if constexpr (TPW == 4) {
      if (four) {
        const int at = (int)(row[0].pos & ((1 << A.c.shift) - 1));
        const int64_t g = kv_slot(A.c, page[0], hh, at);
        uint8_t* pc = A.c.vc + g * (D / 2);
        if constexpr (At::V == 4) {
          *reinterpret_cast<u32x4_t*>(pc + At::v_code(0, lo)) = u32x4_t{wx[0], wx[1], wx[2], wx[3]};
          *reinterpret_cast<u32x4_t*>(pc + At::v_code(0, hi)) = u32x4_t{wy[0], wy[1], wy[2], wy[3]};
        } else {                                           // 2 bytes a token: dimensions lo .. lo + 3, then the next
          auto low = [](uint32_t a, uint32_t b) { return (a & 0xFFFFu) | (b << 16); };
          auto high = [](uint32_t a, uint32_t b) { return (a >> 16) | (b & 0xFFFF0000u); };
          *reinterpret_cast<u32x4_t*>(pc + At::v_code(0, lo)) =
              u32x4_t{low(wx[0], wx[1]), low(wx[2], wx[3]), high(wx[0], wx[1]), high(wx[2], wx[3])};
          *reinterpret_cast<u32x4_t*>(pc + At::v_code(0, hi)) =
              u32x4_t{low(wy[0], wy[1]), low(wy[2], wy[3]), high(wy[0], wy[1]), high(wy[2], wy[3])};
        }
        uint8_t* ps = A.c.vs + g * (D / At::BLK);
        if (first) {
          *reinterpret_cast<uint32_t*>(ps + At::v_scale(0, lo)) = sx[0] | sx[1] << 8 | sx[2] << 16 | sx[3] << 24;
          *reinterpret_cast<uint32_t*>(ps + At::v_scale(0, hi)) = sy[0] | sy[1] << 8 | sy[2] << 16 | sy[3] << 24;
        }
        continue;
      }
    }
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      if (page[i] < 0) continue;
      const int at = (int)(row[i].pos & ((1 << A.c.shift) - 1));
      const int64_t g = kv_slot(A.c, page[i], hh, at & ~3);
      uint8_t* pc = A.c.vc + g * (D / 2);
      if constexpr (At::V == 4) {
        *reinterpret_cast<uint32_t*>(pc + At::v_code(at, lo)) = wx[i];
        *reinterpret_cast<uint32_t*>(pc + At::v_code(at, hi)) = wy[i];
      } else {
        *reinterpret_cast<uint16_t*>(pc + At::v_code(at, lo)) = (uint16_t)wx[i];
        *reinterpret_cast<uint16_t*>(pc + At::v_code(at, lo + 4)) = (uint16_t)(wx[i] >> 16);
        *reinterpret_cast<uint16_t*>(pc + At::v_code(at, hi)) = (uint16_t)wy[i];
        *reinterpret_cast<uint16_t*>(pc + At::v_code(at, hi + 4)) = (uint16_t)(wy[i] >> 16);
      }
      uint8_t* ps = A.c.vs + g * (D / At::BLK);
      if (first) {
        ps[At::v_scale(at, lo)] = (uint8_t)sx[i];
        ps[At::v_scale(at, hi)] = (uint8_t)sy[i];
      }
    }
  }
}

// Reading back: a lane decodes 8 dimensions of TPW tokens in a row, whose loads
// are in flight together. Bound by the bf16 that it writes (8192 tokens of 2 x 32
// heads of 128: 172 MB in 38 us, 4.5 TB/s), or by latency.
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

}  // namespace

hipError_t launch_kv_append(int format, int dim, const KvAppend& a, hipStream_t s) {
  return kv_dispatch(format, dim, [&](auto f, auto d) {
    constexpr int D = decltype(d)::value;
    const int heads = (a.q ? a.q_heads : 0) + (a.k ? 2 * a.c.heads : 0), hpw = 1024 / D;
    auto go = [&](auto f32) {
      constexpr bool F32 = decltype(f32)::value;
      const int64_t wg = grid_of(a.tokens, heads, hpw);
      if (a.b.cu && wg >= kLong)
        kv_append_kernel<decltype(f)::value, D, F32, 4><<<(unsigned)grid_of((a.tokens + 15) / 16 * 4, heads, hpw), 64 * kWaves, 0, s>>>(a);
      else
        kv_append_kernel<decltype(f)::value, D, F32, 1><<<(unsigned)wg, 64 * kWaves, 0, s>>>(a);
    };
    if (a.type == SNIPOP_F32)
      go(std::true_type{});
    else
      go(std::false_type{});
    return hipGetLastError();
  });
}

hipError_t launch_kv_gather(int format, int dim, const KvGather& a, hipStream_t s) {
  return kv_dispatch(format, dim, [&](auto f, auto d) {
    constexpr int D = decltype(d)::value;
    const int heads = (a.k ? a.c.heads : 0) + (a.v ? a.c.heads : 0);
    const int64_t wg = grid_of(a.tokens, heads, 512 / D);
    if (a.b.cu && wg >= kLong)
      kv_gather_kernel<decltype(f)::value, D, 4><<<(unsigned)grid_of((a.tokens + 3) / 4, heads, 512 / D), 64 * kWaves, 0, s>>>(a);
    else
      kv_gather_kernel<decltype(f)::value, D, 1><<<(unsigned)wg, 64 * kWaves, 0, s>>>(a);
    return hipGetLastError();
  });
}

}  // namespace snip
