// Attention of new tokens over a 4-bit key/value cache, gfx950: what the launches
// for few rows (kv_attn.hip) and for prompts (kv_prompt.hip) share.
//
//   s_j = scale q . k_j,  o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m)
//
// in one pass over the keys, with the running maximum m and sum l of a row
// (scores in powers of two: log2 e is part of the scale). The rows of a kv head
// -- the query heads that share it, of one or several tokens -- are taken 16 at a
// time, so that a key is decoded once for all of them:
//   S^T [keys][rows]  = K [keys][dims] . Q^T        (keys are the A operand)
//   O^T [dims][rows] += V^T [dims][keys] . P^T
// A lane holds S^T for one row and 4 + 4 of 32 keys, which is the operand layout
// of P^T when the products run over keys in that order: nothing moves between
// lanes, and the cache's order of bytes gives each lane its keys' dimensions and
// its dimensions' values in one 16-byte load each, 1 KB in a row for the wave.
//
// NVFP4: E2M1 times its E4M3 scale is exact in fp16, and bf16 queries are once a
// power of two puts the row's largest into [2^14, 2^15), as high as fp16 takes it:
// a dimension is exact down to 2^-31 of the largest and below that off by half of
// fp16's last step, 2^-25, which is 2^-39 of the largest at most. MXFP4: exact in
// bf16; the softmax's terms, which bf16 would round to 2^-9, enter in two parts.
#pragma once

#include "kv_common.h"

namespace snip {

namespace {

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef __bf16 b8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4, kRows = 16;
constexpr float kLowest = -3.0e38f;                    // below every score
constexpr int kTop = 15;                               // NVFP4 queries lie below 2^kTop
// A row's m may lag behind its maximum by 2^8, which leaves the output as it is
// for most tiles. NVFP4: it lies 2^7 below the maximum besides, so that terms of
// 2^-21 of the largest keep fp16's precision and 2^-31 still counts: a long
// sequence has many.
constexpr float kLag = 8.0f;
template <int FMT>
constexpr float kLift = FMT == SNIP_NVFP4 ? 7.0f : 0.0f;

template <int FMT, int D>
struct Geo {
  static constexpr bool NV = FMT == SNIP_NVFP4;
  static constexpr int BLK = NV ? 16 : 32;
  static constexpr int PB = kv_key_piece(D), VB = kv_value_piece(D), SB = kv_scale_piece(D, BLK);
  static constexpr int KL = D / 2 / PB / 4;            // a lane's loads of keys (16 tokens)
  static constexpr int VL = D / 2 / VB / 16;           // of values (4 of 16 tokens)
  static constexpr int KD = PB / 4;                    // dwords of a key's piece: products over 32 dimensions
  static constexpr int DT = D / 16;                    // tiles of 16 dimensions of O^T
};

// What a lane holds of 32 tokens.
template <int FMT, int D>
struct Tile {
  using G = Geo<FMT, D>;
  uint32_t k[2][G::KL][G::KD], ks[2][G::KL];
  uint32_t v[2][G::VL][G::VB], vs[2][G::VL];
};

template <bool NT, typename T>
__device__ __forceinline__ T fetch(const uint8_t* p) {
  const T* q = reinterpret_cast<const T*>(p);
  return NT ? __builtin_nontemporal_load(q) : *q;
}

template <bool NT, int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const u32x4_t x = fetch<NT, u32x4_t>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x[i];
  } else {
    static_assert(N == 2, "");
    const u32x2_t x = fetch<NT, u32x2_t>(p);
    w[0] = x[0];
    w[1] = x[1];
  }
}

// 16 tokens from `slot` (wave-uniform): a lane's share.
template <int FMT, int D, bool NT = false>
__device__ __forceinline__ void load_half(const KvCache& C, int64_t slot, uint32_t (&k)[Geo<FMT, D>::KL][Geo<FMT, D>::KD],
                                          uint32_t (&ksc)[Geo<FMT, D>::KL], uint32_t (&v)[Geo<FMT, D>::VL][Geo<FMT, D>::VB],
                                          uint32_t (&vsc)[Geo<FMT, D>::VL]) {
  using G = Geo<FMT, D>;
  const uint32_t lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4;   // unsigned: added to scalar bases by the loads
  const uint8_t* kc = C.kc + slot * (D / 2);
  const uint8_t* ks = C.ks + slot * (D / G::BLK);
  const uint8_t* vc = C.vc + slot * (D / 2);
  const uint8_t* vs = C.vs + slot * (D / G::BLK);
#pragma unroll
  for (int l = 0; l < G::KL; ++l) {
    load_words<NT>(kc + (64 * l + lane) * G::PB, k[l]);
    if constexpr (G::SB == 2)
      ksc[l] = *reinterpret_cast<const uint16_t*>(ks + (64 * l + lane) * 2);
    else if constexpr (2 * G::PB < G::BLK)             // two pieces to a block
      ksc[l] = ks[c / 2 * 16 + n];
    else
      ksc[l] = ks[64 * l + lane];
  }
#pragma unroll
  for (int l = 0; l < G::VL; ++l) {
    load_words<NT>(vc + c * 2 * D + (16 * l + n) * 4 * G::VB, v[l]);
    vsc[l] = *reinterpret_cast<const uint32_t*>(vs + c * 4 * (D / G::BLK) + (16 * l + n) * 2 * G::VB / G::BLK * 4);
  }
}

__device__ __forceinline__ uint32_t bits(h2_t v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ uint32_t bits(bf16x2_t v) { return __builtin_bit_cast(uint32_t, v); }

template <int J>
__device__ __forceinline__ h2_t fp16_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, J);
}

// E8M0 byte as the scale operand of a conversion, which takes its exponent.
__device__ __forceinline__ float e8m0_val(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FC00000u : b << 23);
}

// 8 dimensions of a key: the A operand of a product over 32 dimensions.
template <int FMT>
__device__ __forceinline__ u32x4_t decode_key(uint32_t w, h2_t s, float e) {
  if constexpr (FMT == SNIP_NVFP4) {
    return u32x4_t{bits(fp16_pair<0>(w) * s), bits(fp16_pair<1>(w) * s), bits(fp16_pair<2>(w) * s), bits(fp16_pair<3>(w) * s)};
  } else {
    return u32x4_t{bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, e, 0)), bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, e, 1)),
                   bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, e, 2)), bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, e, 3))};
  }
}

template <int FMT>
__device__ __forceinline__ f4_t mfma(u32x4_t a, u32x4_t b, f4_t c) {
  if constexpr (FMT == SNIP_NVFP4)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, a), __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8_t, a), __builtin_bit_cast(b8_t, b), c, 0, 0, 0);
}

// Maximum and sum over the four lanes of a row, in each of them.
__device__ __forceinline__ float row_max(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t x = __float_as_uint(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
  const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float row_sum(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t x = __float_as_uint(__uint_as_float(r[0]) + __uint_as_float(r[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// The values of 4 tokens at a lane's 2 VB dimensions (of load l), as pairs of
// tokens: out[i][p] is dimension i of tokens 2p and 2p + 1, times their scales.
template <int FMT, int D>
__device__ __forceinline__ void decode_values(const uint32_t (&w)[Geo<FMT, D>::VB], uint32_t sc,
                                              uint32_t (&out)[2 * Geo<FMT, D>::VB][2]) {
  constexpr int VB = Geo<FMT, D>::VB;
  if constexpr (FMT == SNIP_NVFP4) {
    const h2_t s[2] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sc, 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sc, 1.0f, true)};
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if constexpr (VB == 4) {                         // tokens 2p, 2p + 1: codes of even and of odd dimensions side by side
        const uint32_t a = w[2 * p], b = w[2 * p + 1];
        const uint32_t ev = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), od = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
        out[0][p] = bits(fp16_pair<0>(ev) * s[p]);
        out[1][p] = bits(fp16_pair<0>(od) * s[p]);
        out[2][p] = bits(fp16_pair<1>(ev) * s[p]);
        out[3][p] = bits(fp16_pair<1>(od) * s[p]);
        out[4][p] = bits(fp16_pair<2>(ev) * s[p]);
        out[5][p] = bits(fp16_pair<2>(od) * s[p]);
        out[6][p] = bits(fp16_pair<3>(ev) * s[p]);
        out[7][p] = bits(fp16_pair<3>(od) * s[p]);
      } else {                                         // a word has both tokens: 4 dimensions each
        const uint32_t a = w[p], b = a >> 16;
        const uint32_t ev = (a & 0x0F0Fu) | ((b << 4) & 0xF0F0u), od = ((a >> 4) & 0x0F0Fu) | (b & 0xF0F0u);
        out[0][p] = bits(fp16_pair<0>(ev) * s[p]);
        out[1][p] = bits(fp16_pair<0>(od) * s[p]);
        out[2][p] = bits(fp16_pair<1>(ev) * s[p]);
        out[3][p] = bits(fp16_pair<1>(od) * s[p]);
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float ea = e8m0_val((sc >> (16 * p)) & 0xFFu), eb = e8m0_val((sc >> (16 * p + 8)) & 0xFFu);
      const uint32_t a = VB == 4 ? w[2 * p] : w[p], b = VB == 4 ? w[2 * p + 1] : w[p] >> 16;
      auto pair = [&](uint32_t x, uint32_t y, int j) {   // dimensions 2j, 2j + 1 of both tokens
        out[2 * j][p] = __builtin_amdgcn_perm(y, x, 0x05040100u);
        out[2 * j + 1][p] = __builtin_amdgcn_perm(y, x, 0x07060302u);
      };
      pair(bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, ea, 0)), bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(b, eb, 0)), 0);
      pair(bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, ea, 1)), bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(b, eb, 1)), 1);
      if constexpr (VB == 4) {
        pair(bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, ea, 2)), bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(b, eb, 2)), 2);
        pair(bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, ea, 3)), bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(b, eb, 3)), 3);
      }
    }
  }
}

// A wave's share of 16 rows: queries, running maximum, sum and output.
template <int FMT, int D>
struct Rows {
  using G = Geo<FMT, D>;
  u32x4_t q[G::KL][G::KD];
  float factor;                // of a score, to powers of two
  int first, last;             // keys that this lane's row sees
  float m, l;                  // l: of this lane's keys
  f4_t o[G::DT];

  // The row's head (qp null: no row) is asked for here, and made the products'
  // operand in start().
  __device__ __forceinline__ void load(const uint16_t* qp) {
    const int c = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int l_ = 0; l_ < G::KL; ++l_)
#pragma unroll
      for (int w = 0; w < G::KD; ++w)
        q[l_][w] = qp ? *reinterpret_cast<const u32x4_t*>(qp + (c + 4 * l_) * 2 * G::PB + 8 * w) : u32x4_t{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void start(float scale, int ek) {
    factor = scale;
    if constexpr (G::NV) {
      float big = 0.0f;
#pragma unroll
      for (int l_ = 0; l_ < G::KL; ++l_)
#pragma unroll
        for (int w = 0; w < G::KD; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) big = fmaxf(big, fmaxf(fabsf(bf16_lo(q[l_][w][i])), fabsf(bf16_hi(q[l_][w][i]))));
      big = row_max(big);
      int e;
      frexpf(big, &e);
      e = big < __builtin_inff() ? e - kTop : 0;
#pragma unroll
      for (int l_ = 0; l_ < G::KL; ++l_)
#pragma unroll
        for (int w = 0; w < G::KD; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            q[l_][w][i] = bits(h2_t{(_Float16)ldexpf(bf16_lo(q[l_][w][i]), -e), (_Float16)ldexpf(bf16_hi(q[l_][w][i]), -e)});
      factor = ldexpf(scale, e + ek);
    }
    m = kLowest;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < G::DT; ++i) o[i] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
};

struct Span {                  // of one sequence
  int64_t row0, pos0;          // first row in the call's matrices, its position
  int rows;                    // (token, query head) pairs of a kv head
  int tiles, steps;            // units a head, steps a unit
  int keys;                    // from the first that its first row sees to the last row's
};

__device__ __forceinline__ int limit(const KvAttn& A, int64_t p) {
  return (int)(p < 0 ? -1 : p >= A.b.max_len ? A.b.max_len - 1 : p);
}
// First key that a row at position p sees; the table's end where its window lies
// behind that.
__device__ __forceinline__ int first_key(const KvAttn& A, int64_t p) {
  if (!A.window || p < A.window) return 0;
  return (int)(p - A.window + 1 < A.b.max_len ? p - A.window + 1 : A.b.max_len);
}

__device__ __forceinline__ Span span_of(const KvAttn& A, int b, int unit_rows) {
  Span x = {};
  if (b >= A.b.seqs) return x;
  int64_t a = b, e = b + 1;
  if (A.b.cu) {
    a = entries(A.b.cu)[b];
    e = entries(A.b.cu)[b + 1];
  }
  const int64_t len = entries(A.b.lens)[b];
  x.row0 = a;
  x.pos0 = len - (e - a);
  if (e > A.tokens) e = A.tokens;
  if (a < 0 || e <= a) return x;
  x.rows = (int)(e - a) * A.group;
  x.tiles = (x.rows + unit_rows - 1) / unit_rows;
  x.keys = limit(A, len - 1) + 1 - (first_key(A, x.pos0) & ~31);
  x.steps = x.keys > A.step ? (x.keys + A.step - 1) / A.step : 1;   // a unit without keys writes its zeros
  return x;
}

// Whether the launch for prompts has a sequence, where there are both.
__device__ __forceinline__ bool prompt_rows(const KvAttn& A, const Span& x) {
  return x.rows > (x.keys > A.far ? A.some : A.few);
}

// An output: the values' power of two after the quotient, since 2^ev / L may lie
// below fp32's normal range where the output does not.
template <int FMT>
__device__ __forceinline__ float output(float o, float inv, int ev) {
  return FMT == SNIP_NVFP4 ? ldexpf(o * inv, ev) : o * inv;
}

__device__ __forceinline__ void store_lse(const KvAttn& A, int64_t t, int qh, float M, float L) {
  A.lse[t * A.q_heads + qh] = L == 0.0f ? -__builtin_inff() : (M + __builtin_amdgcn_logf(L)) * 0.693147180559945309f;
}

}  // namespace

}  // namespace snip
