// Attention of new tokens over a 4-bit key/value cache, gfx950.
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
// NVFP4: E2M1 times its E4M3 scale is exact in fp16, and bf16 queries are once
// the row's power of two is taken out (dimensions 2^-14 below the row's largest
// lose bits of 2^-25 of it). MXFP4: exact in bf16; the softmax's terms, which
// bf16 would round to 2^-9, enter in two parts.
#include "kv_common.h"

namespace snip {

namespace {

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef __bf16 b8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4, kRows = 16;
constexpr float kLowest = -3.0e38f;                    // below every score

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

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x[i];
  } else {
    static_assert(N == 2, "");
    const u32x2_t x = *reinterpret_cast<const u32x2_t*>(p);
    w[0] = x[0];
    w[1] = x[1];
  }
}

// 16 tokens from `slot` (wave-uniform) into half `h` of a tile.
template <int FMT, int D>
__device__ __forceinline__ void load_half(const KvCache& C, int64_t slot, int h, Tile<FMT, D>& T) {
  using G = Geo<FMT, D>;
  const int lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4;
  const uint8_t* kc = C.kc + slot * (D / 2);
  const uint8_t* ks = C.ks + slot * (D / G::BLK);
  const uint8_t* vc = C.vc + slot * (D / 2);
  const uint8_t* vs = C.vs + slot * (D / G::BLK);
#pragma unroll
  for (int l = 0; l < G::KL; ++l) {
    load_words<G::KD>(kc + (64 * l + lane) * G::PB, T.k[h][l]);
    if constexpr (G::SB == 2)
      T.ks[h][l] = *reinterpret_cast<const uint16_t*>(ks + (64 * l + lane) * 2);
    else if constexpr (2 * G::PB < G::BLK)             // two pieces to a block
      T.ks[h][l] = ks[c / 2 * 16 + n];
    else
      T.ks[h][l] = ks[64 * l + lane];
  }
#pragma unroll
  for (int l = 0; l < G::VL; ++l) {
    load_words<G::VB>(vc + c * 2 * D + (16 * l + n) * 4 * G::VB, T.v[h][l]);
    T.vs[h][l] = *reinterpret_cast<const uint32_t*>(vs + c * 4 * (D / G::BLK) + (16 * l + n) * 2 * G::VB / G::BLK * 4);
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

  // qp: the row's head (or null: no row).
  __device__ __forceinline__ void start(const uint16_t* qp, float scale, int ek) {
    const int c = (threadIdx.x & 63) >> 4;
    float big = 0.0f;
#pragma unroll
    for (int l_ = 0; l_ < G::KL; ++l_)
#pragma unroll
      for (int w = 0; w < G::KD; ++w) {
        q[l_][w] = qp ? *reinterpret_cast<const u32x4_t*>(qp + (c + 4 * l_) * 2 * G::PB + 8 * w) : u32x4_t{0u, 0u, 0u, 0u};
        if constexpr (G::NV) {
#pragma unroll
          for (int i = 0; i < 4; ++i) big = fmaxf(big, fmaxf(fabsf(bf16_lo(q[l_][w][i])), fabsf(bf16_hi(q[l_][w][i]))));
        }
      }
    factor = scale;
    if constexpr (G::NV) {
      int e;
      frexpf(row_max(big), &e);
      const bool finite = row_max(big) < __builtin_inff();
      e = finite ? e : 0;
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

// Scores of 32 keys for 16 rows: s[half][j] is key 16 half + 4 c + j.
template <int FMT, int D>
__device__ __forceinline__ void scores(const Tile<FMT, D>& T, const Rows<FMT, D>& R, f4_t (&s)[2]) {
  using G = Geo<FMT, D>;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    s[h] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int l = 0; l < G::KL; ++l) {
      h2_t sc = {};
      float e = 0.0f;
      if constexpr (G::NV)
        sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(T.ks[h][l], 1.0f, false);
      else
        e = e8m0_val(T.ks[h][l]);
#pragma unroll
      for (int w = 0; w < G::KD; ++w) {
        const int b = G::SB == 2 ? w / 2 : 0;          // block of the piece
        s[h] = mfma<FMT>(decode_key<FMT>(T.k[h][l][w], h2_t{sc[b], sc[b]}, e), R.q[l][w], s[h]);
      }
    }
  }
}

// Work is counted in steps: the workgroup's waves take 32 keys each. A unit --
// 16 rows of one kv head of one sequence -- has the steps of the sequence's
// keys, units follow each other by sequence, head and rows, and the steps of the
// call are shared evenly among the workgroups, whatever the lengths. A workgroup
// finds its share from lens and cu alone, so a captured launch follows them.
constexpr int kStep = 32 * kWaves;

struct Span {                  // of one sequence
  int64_t row0, pos0;          // first row in the call's matrices, its position
  int rows;                    // (token, query head) pairs of a kv head
  int tiles, steps;            // units a head, steps a unit
};

__device__ __forceinline__ int limit(const KvAttn& A, int64_t p) {
  return (int)(p < 0 ? -1 : p >= A.b.max_len ? A.b.max_len - 1 : p);
}
// First key that a row at position p sees.
__device__ __forceinline__ int first_key(const KvAttn& A, int64_t p) {
  return A.window && p >= A.window ? limit(A, p - A.window + 1) : 0;
}

__device__ __forceinline__ Span span_of(const KvAttn& A, int b) {
  Span x = {};
  if (b >= A.b.seqs) return x;
  int64_t a = b, e = b + 1;
  if (A.b.cu) {
    a = A.b.cu[b];
    e = A.b.cu[b + 1];
  }
  const int64_t len = A.b.lens[b];
  x.row0 = a;
  x.pos0 = len - (e - a);
  if (e > A.tokens) e = A.tokens;
  if (a < 0 || e <= a) return x;
  x.rows = (int)(e - a) * A.group;
  x.tiles = (x.rows + kRows - 1) / kRows;
  const int n = limit(A, len - 1) + 1 - (first_key(A, x.pos0) & ~31);
  x.steps = n > kStep ? (n + kStep - 1) / kStep : 1;   // a unit without keys writes its zeros
  return x;
}

__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// The sequences 64 at a time: the steps up to and with each of them, in the
// wave's own LDS (a register each would cost the kernel a wave of occupancy).
struct Cursor {
  int64_t* upto;               // [64]
  int seq0;
  int64_t before, end;         // steps before the 64, and with them

  __device__ __forceinline__ void load(const KvAttn& A, int s0, int64_t b) {
    const int lane = threadIdx.x & 63;
    const Span x = span_of(A, s0 + lane);
    int64_t n = (int64_t)x.tiles * x.steps * A.c.heads;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t v = __shfl_up(n, o, 64);
      if (lane >= o) n += v;
    }
    seq0 = s0;
    before = b;
    end = uniform(b + __shfl(n, 63, 64));
    upto[lane] = b + n;
    __builtin_amdgcn_wave_barrier();
  }
  // Steps of all sequences; leaves the cursor at the first ones.
  __device__ __forceinline__ int64_t total(const KvAttn& A) {
    load(A, 0, 0);
    if (A.b.seqs <= 64) return end;
    for (int s = 64; s < A.b.seqs; s += 64) load(A, s, end);
    const int64_t n = end;
    load(A, 0, 0);
    return n;
  }
  // The sequence that step `at` is in, and the steps before it.
  __device__ __forceinline__ int seek(const KvAttn& A, int64_t at, int64_t* from) {
    while (at >= end) load(A, seq0 + 64, end);
    const int i = __ffsll((unsigned long long)__ballot(upto[threadIdx.x & 63] > at)) - 1;
    *from = i ? uniform(upto[i - 1]) : before;
    return seq0 + i;
  }
};

// The steps of n workgroups: q each, one more for the first r.
struct Shares {
  int64_t q, r;
  __device__ __forceinline__ Shares(int64_t total, int n) {
    if (total >> 31) {
      q = total / n;
    } else {
      q = (uint32_t)total / (uint32_t)n;
    }
    r = total - q * n;
  }
  __device__ __forceinline__ int64_t first(int w) const { return w * q + (w < r ? w : r); }
  __device__ __forceinline__ int owner(int64_t at) const {   // of a step
    const int64_t many = r * (q + 1);
    if (at < many) return at >> 31 ? (int)(at / (q + 1)) : (int)((uint32_t)at / (uint32_t)(q + 1));
    const int64_t rest = at - many;
    return (int)r + (rest >> 31 ? (int)(rest / q) : (int)((uint32_t)rest / (uint32_t)q));
  }
};

}  // namespace

// What a workgroup leaves for the joining launch: two slots, of the unit that
// its share begins within and of the one that it ends within (16 maxima, 16
// sums, 16 rows of output each), and where the latter's output belongs.
struct Left {
  int64_t row0;                // first row of the sequence
  int rows, r0, head;          // rows of the unit (0: none is left), its first, its kv head
  int last;                    // the workgroup that has the unit's last step
};

namespace {

constexpr int slot_floats(int dim) { return kRows * (dim + 2); }

template <int FMT, int D>
__global__ __launch_bounds__(64 * kWaves, 3) void kv_attn_kernel(KvAttn A) {
  using G = Geo<FMT, D>;
  constexpr int LD = D + 4;                            // a row in LDS: the lanes' rows meet different banks
  __shared__ float stats[2][kWaves][kRows];
  __shared__ float part[kWaves][kRows * LD];
  const int lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int ek = 0, ev = 0;
  if constexpr (G::NV) {
    ek = A.c.texp[0];
    ev = A.c.texp[1];
  }
  __shared__ int64_t upto[kWaves][64];
  Cursor cur;
  cur.upto = upto[wave];
  const int64_t total = cur.total(A);
  const Shares shares(total, gridDim.x);
  int64_t at = shares.first(blockIdx.x);
  const int64_t stop = shares.first(blockIdx.x + 1);
  Left left = {0, 0, 0, 0, 0};
  while (at < stop) {
  int64_t from;
  const int seq = cur.seek(A, at, &from);
  const Span U = span_of(A, seq);
  const int64_t rel = at - from;
  const int unit = rel >> 31 ? (int)(rel / U.steps) : (int)((uint32_t)rel / (uint32_t)U.steps);
  const int s0 = (int)(rel - (int64_t)unit * U.steps);
  const int s1 = stop - at < U.steps - s0 ? s0 + (int)(stop - at) : U.steps;
  at += s1 - s0;
  const int head = unit / U.tiles, r0 = unit % U.tiles * kRows;
  const int rows = U.rows - r0 < kRows ? U.rows - r0 : kRows;
  Rows<FMT, D> R;
  const int r = r0 + n, tok = r / A.group;
  const bool mine = n < rows;
  R.start(mine ? A.q + (U.row0 + tok) * A.ldq + (int64_t)(head * A.group + r % A.group) * D : nullptr, A.scale, ek);
  // keys of this lane's row, of any row of the unit and of all
  const int64_t p0 = U.pos0 + r0 / A.group, p1 = U.pos0 + (r0 + rows - 1) / A.group;
  R.last = mine ? limit(A, U.pos0 + tok) : -1;
  R.first = first_key(A, U.pos0 + tok);
  const int first = first_key(A, p0), every_first = first_key(A, p1), every_last = limit(A, p0);
  const int begin = (first_key(A, U.pos0) & ~31) + s0 * kStep;
  const int last = s1 == U.steps ? limit(A, p1) : (begin + (s1 - s0) * kStep - 1 < limit(A, p1) ? begin + (s1 - s0) * kStep - 1 : limit(A, p1));
  // The table's entries are asked for two steps ahead, as scalars of the constant
  // address space: a vector load would be waited for in order with the keys'.
  struct Pages {
    int p[2];
  };
  typedef const __attribute__((address_space(4))) int32_t* Entries;
  const Entries entries = (Entries)(uintptr_t)(A.b.table + (int64_t)seq * A.b.table_ld);
  auto pages = [&](int key) {
    Pages g;
#pragma unroll
    for (int h = 0; h < 2; ++h) g.p[h] = entries[(key + 16 * h < last ? key + 16 * h : last) >> A.c.shift];
    return g;
  };
  auto mapped = [&](const Pages& g, int h) { return (uint32_t)g.p[h] < (uint32_t)A.c.pages; };
  // Loads are never skipped, since the wait for a tile counts those of the next
  // one: beyond the last key, and where a page is not mapped, they read others.
  auto load = [&](int key, const Pages& g, Tile<FMT, D>& T) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      load_half<FMT, D>(A.c, kv_slot(A.c, mapped(g, h) ? g.p[h] : 0, head, (key + 16 * h) & ((1 << A.c.shift) - 1)), h, T);
  };
  auto use = [&](int key, const Pages& g, Tile<FMT, D>& T) {
    f4_t s[2];
    scores<FMT, D>(T, R, s);
    const bool whole = mapped(g, 0) & mapped(g, 1) & (key >= every_first) & (key + 31 <= every_last);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[h][j] *= R.factor;
    if (!whole) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k0 = key + 16 * h + 4 * c, end = mapped(g, h) ? last : -1, mine_end = R.last < end ? R.last : end;
        uint32_t keep = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[h][j] = (k0 + j >= R.first) & (k0 + j <= mine_end) ? s[h][j] : -__builtin_inff();
          keep |= (k0 + j >= first) & (k0 + j <= end) ? 0xFFu << (8 * j) : 0u;
        }
        // values of places that no row sees may be anything: their scales are replaced
#pragma unroll
        for (int l = 0; l < G::VL; ++l) T.vs[h][l] &= keep;
      }
    }
    float top = kLowest;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, s[h][j]);
    // the maximum may lag by 2^8: terms of up to 256 are as exact, and most tiles leave the output as it is
    if (__any(top > R.m + 8.0f)) {
      top = fmaxf(row_max(top), R.m);
      const float f = __builtin_amdgcn_exp2f(R.m - top);
      R.m = top;
      R.l *= f;
#pragma unroll
      for (int i = 0; i < G::DT; ++i) R.o[i] *= f;
    }
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(s[i / 4][i % 4] - R.m);
      R.l += p[i];
    }
    u32x4_t ph, pl;                                    // fp16, or the two parts in bf16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (G::NV) {
        ph[i] = bits(h2_t{(_Float16)p[2 * i], (_Float16)p[2 * i + 1]});
      } else {
        ph[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
        pl[i] = pack_bf16(p[2 * i] - bf16_lo(ph[i]), p[2 * i + 1] - bf16_hi(ph[i]));
      }
    }
#pragma unroll
    for (int l = 0; l < G::VL; ++l) {
      uint32_t v0[2 * G::VB][2], v1[2 * G::VB][2];
      decode_values<FMT, D>(T.v[0][l], T.vs[0][l], v0);
      decode_values<FMT, D>(T.v[1][l], T.vs[1][l], v1);
#pragma unroll
      for (int i = 0; i < 2 * G::VB; ++i) {
        const u32x4_t a = {v0[i][0], v0[i][1], v1[i][0], v1[i][1]};
        f4_t& o = R.o[l * 2 * G::VB + i];
        o = mfma<FMT>(a, ph, o);
        if constexpr (!G::NV) o = mfma<FMT>(a, pl, o);
      }
    }
  };
  int key = begin + 32 * wave;
  Tile<FMT, D> T0, T1;
  if (key <= last) {
    Pages g0 = pages(key), g1 = pages(key + kStep);
    load(key, g0, T0);
    while (true) {
      load(key + kStep, g1, T1);
      const Pages g2 = pages(key + 2 * kStep);
      use(key, g0, T0);
      key += kStep;
      if (key > last) break;
      load(key + kStep, g2, T0);
      const Pages g3 = pages(key + 2 * kStep);
      use(key, g1, T1);
      key += kStep;
      if (key > last) break;
      g0 = g2;
      g1 = g3;
    }
  }

  // the waves' shares of the rows, joined
  const float l = row_sum(R.l);
  if (c == 0) {
    stats[0][wave][n] = R.m;
    stats[1][wave][n] = l;
  }
#pragma unroll
  for (int i = 0; i < G::DT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)                        // dimension of O^T's row 4 c + j in tile i
      part[wave][n * LD + (i / (2 * G::VB)) * 32 * G::VB + (4 * c + j) * 2 * G::VB + i % (2 * G::VB)] = R.o[i][j];
  __syncthreads();
  const int row = threadIdx.x / 16, d0 = threadIdx.x % 16 * (D / 16);
  float M = kLowest, L = 0.0f, w[kWaves];
#pragma unroll
  for (int i = 0; i < kWaves; ++i) M = fmaxf(M, stats[0][i][row]);
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    w[i] = __builtin_amdgcn_exp2f(stats[0][i][row] - M);
    L += stats[1][i][row] * w[i];
  }
  if (row < rows) {
    const bool all = s1 - s0 == U.steps;               // the unit's: the output; else a slot, the first of a share
    const int rr = r0 + row;                           // where it goes on with a unit, the second where it leaves one
    const int64_t t = U.row0 + rr / A.group;
    const int qh = head * A.group + rr % A.group;
    float* slot = A.part + (2 * (int64_t)blockIdx.x + (s0 == 0)) * slot_floats(D);
    const float inv = !all ? 1.0f : L == 0.0f ? 0.0f : ldexpf(1.0f / L, ev);
#pragma unroll
    for (int d = 0; d < D / 16; d += 4) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) x[e] += part[i][row * LD + d0 + d + e] * w[i];
        x[e] *= inv;
      }
      if (all)
        store_whole(A.out, false, t * A.ldo + (int64_t)qh * D + d0 + d, x);
      else
        store_whole(slot, true, 2 * kRows + row * D + d0 + d, x);
    }
    if (d0 == 0) {
      if (!all) {
        slot[row] = M;
        slot[kRows + row] = L;
      } else if (A.lse) {
        A.lse[t * A.q_heads + qh] = L == 0.0f ? -__builtin_inff() : (M + __builtin_amdgcn_logf(L)) * 0.693147180559945309f;
      }
    }
  }
  if (s0 == 0 && s1 < U.steps) left = Left{U.row0, rows, r0, head, shares.owner(at - s1 + U.steps - 1)};
  if (at < stop) __syncthreads();
  }
  if (threadIdx.x == 0) A.left[blockIdx.x] = left;
}

// A unit that several workgroups had a share of, joined: blockIdx.x is the one
// that has its first step, blockIdx.y the row. The parts are taken by several
// groups of lanes and added in a fixed order.
template <int D>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttn A, bool nv) {
  constexpr int LR = D / 4, SUBS = 256 / LR;           // lanes of a row, parts taken at once
  __shared__ float sm[SUBS], sl[SUBS];
  __shared__ f4_t so[SUBS][LR];
  const int w0 = blockIdx.x, row = blockIdx.y;
  const Left U = A.left[w0];
  if (row >= U.rows) return;
  const int w1 = U.last;
  auto slot = [&](int w) { return A.part + (2 * (int64_t)w + (w == w0)) * slot_floats(D); };
  const int sub = threadIdx.x / LR, d = threadIdx.x % LR * 4;
  float M = kLowest, L = 0.0f;
  f4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int w = w0 + sub; w <= w1; w += SUBS) M = fmaxf(M, slot(w)[row]);
#pragma unroll 4
  for (int w = w0 + sub; w <= w1; w += SUBS) {
    const float* p = slot(w);
    const float f = __builtin_amdgcn_exp2f(p[row] - M);
    L += p[kRows + row] * f;
    x += *reinterpret_cast<const f4_t*>(p + 2 * kRows + row * D + d) * f;
  }
  so[sub][threadIdx.x % LR] = x;
  if (d == 0) {
    sm[sub] = M;
    sl[sub] = L;
  }
  __syncthreads();
  if (sub) return;
  M = kLowest;
  L = 0.0f;
  x = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < SUBS; ++i) M = fmaxf(M, sm[i]);
#pragma unroll
  for (int i = 0; i < SUBS; ++i) {
    const float f = __builtin_amdgcn_exp2f(sm[i] - M);
    L += sl[i] * f;
    x += so[i][threadIdx.x] * f;
  }
  const int rr = U.r0 + row;
  const int64_t t = U.row0 + rr / A.group;
  const int qh = U.head * A.group + rr % A.group;
  const float inv = L == 0.0f ? 0.0f : ldexpf(1.0f / L, nv ? A.c.texp[1] : 0);
  const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
  store_whole(A.out, false, t * A.ldo + (int64_t)qh * D + d, y);
  if (A.lse && d == 0)
    A.lse[t * A.q_heads + qh] = L == 0.0f ? -__builtin_inff() : (M + __builtin_amdgcn_logf(L)) * 0.693147180559945309f;
}

}  // namespace

// Workgroups of the split kernel: as many as are resident.
constexpr int workers_of(int dim) { return dim == 64 ? 1024 : dim == 128 ? 768 : 256; }

int64_t kv_attn_tiles(int64_t tokens, int64_t seqs, int64_t group, bool cu) {
  return cu ? tokens * group / kRows + seqs : tokens * ((group + kRows - 1) / kRows);
}

size_t kv_attn_slots(int dim) {
  return (size_t)workers_of(dim) * (2 * slot_floats(dim) * sizeof(float) + sizeof(Left));
}


hipError_t launch_kv_attn(int format, int dim, KvAttn a, hipStream_t s) {
  a.left = reinterpret_cast<Left*>(a.part + (size_t)workers_of(dim) * 2 * slot_floats(dim));
  auto go = [&](auto f, auto d) {
    constexpr int D = decltype(d)::value;
    kv_attn_kernel<decltype(f)::value, D><<<workers_of(D), 64 * kWaves, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t rows = a.b.cu ? kRows : a.group;     // a unit has no more
    kv_join_kernel<D><<<dim3(workers_of(D) - 1, rows < kRows ? rows : kRows), 256, 0, s>>>(a, format == SNIP_NVFP4);
    return hipGetLastError();
  };
  auto of = [&](auto f) {
    return dim == 64    ? go(f, std::integral_constant<int, 64>{})
           : dim == 128 ? go(f, std::integral_constant<int, 128>{})
                        : go(f, std::integral_constant<int, 256>{});
  };
  return format == SNIP_NVFP4 ? of(std::integral_constant<int, SNIP_NVFP4>{})
                              : of(std::integral_constant<int, SNIP_MXFP4>{});
}

}  // namespace snip
