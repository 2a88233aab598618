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
      e = big < __builtin_inff() ? e : 0;
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

// Work is counted in steps of a number of keys. A unit -- 16 R rows of one kv
// head of one sequence -- has the steps of the sequence's keys, units follow each
// other by sequence, head and rows, and the steps of the call are shared evenly
// among the workgroups, whatever the lengths. A workgroup finds its share from
// lens and cu alone, so a captured launch follows them.
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
  const int n = limit(A, len - 1) + 1 - (first_key(A, x.pos0) & ~31);
  x.steps = n > A.step ? (n + A.step - 1) / A.step : 1;   // a unit without keys writes its zeros
  return x;
}

// Sum over the lanes up to and with each.
__device__ __forceinline__ int wave_prefix(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // the rows before: row_bcast 15, 31
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// Finds the sequence of a step. The sequences are taken in 64 groups of
// neighbours, a group a lane, so that all loads of lens are in flight at once;
// the steps up to and with each group, and with each of 64 sequences of the group
// that was looked into last, lie in the wave's own LDS (registers would cost the
// kernel a wave of occupancy).
struct Cursor {
  int* coarse;                 // [64]
  int* fine;                   // [64]
  int unit_rows, each;         // sequences of a group
  int seq0, before, end;       // the 64 looked into last: the first, the steps before and with them

  __device__ __forceinline__ int cost(const KvAttn& A, int b) const {
    const Span x = span_of(A, b, unit_rows);
    return A.split && x.rows > A.few ? 0 : x.tiles * x.steps * A.c.heads;
  }
  // Steps of all sequences.
  __device__ __forceinline__ int total(const KvAttn& A) {
    const int lane = threadIdx.x & 63;
    each = (A.b.seqs + 63) >> 6;
    int n = 0;
#pragma unroll 4
    for (int j = 0; j < each; ++j) n += cost(A, lane * each + j);
    n = wave_prefix(n);
    coarse[lane] = n;
    before = end = 0;
    __builtin_amdgcn_wave_barrier();
    return __builtin_amdgcn_readlane(n, 63);
  }
  // The sequence that step `at` is in, and the steps before it.
  __device__ __forceinline__ int seek(const KvAttn& A, int at, int* from) {
    const int lane = threadIdx.x & 63;
    if (each > 1 && (at < before || at >= end)) {
      const int g = __ffsll((unsigned long long)__ballot(coarse[lane] > at)) - 1;
      before = g ? __builtin_amdgcn_readfirstlane(coarse[g - 1]) : 0;
      for (int o = 0;; o += 64) {
        seq0 = g * each + o;
        const int n = before + wave_prefix(o + lane < each ? cost(A, seq0 + lane) : 0);
        end = __builtin_amdgcn_readlane(n, 63);
        if (at < end || o + 64 >= each) {
          fine[lane] = n;
          break;
        }
        before = end;
      }
      __builtin_amdgcn_wave_barrier();
    }
    const int* upto = each > 1 ? fine : coarse;
    const int i = __ffsll((unsigned long long)__ballot(upto[lane] > at)) - 1;
    *from = i ? __builtin_amdgcn_readfirstlane(upto[i - 1]) : each > 1 ? before : 0;
    return (each > 1 ? seq0 : 0) + i;
  }
};

// The steps of n workgroups: q each, one more for the first r.
struct Shares {
  uint32_t q, r;
  __device__ __forceinline__ Shares(uint32_t total, uint32_t n) : q(total / n), r(total % n) {}
  __device__ __forceinline__ int first(uint32_t w) const { return (int)(w * q + (w < r ? w : r)); }
  __device__ __forceinline__ int owner(uint32_t at) const {   // of a step
    const uint32_t many = r * (q + 1);
    return (int)(at < many ? at / (q + 1) : r + (at - many) / q);
  }
};

}  // namespace

// What a workgroup leaves for the joining launch: two slots, of the unit that
// its share begins within and of the one that it ends within (maxima, sums and
// rows of output), and where the latter's output belongs.
struct Left {
  int64_t row0;                // first row of the sequence
  int rows, r0, head;          // rows of the unit (0: none is left), its first, its kv head
  int last;                    // the workgroup that has the unit's last step
};

namespace {

constexpr int slot_floats(int dim, int rows) { return rows * (dim + 2); }

// Row tiles of a unit, waves of a SIMD that the registers are held to, and
// workgroups: as many as are resident.
constexpr int most_tiles(int dim) { return dim == 256 ? 1 : 2; }
constexpr int waves_of(int dim, int tiles) { return dim == 256 ? 2 : (dim == 128 ? 3 : 4) - (tiles == 2); }
constexpr int workers_of(int dim, int tiles) { return 256 * waves_of(dim, tiles); }

__device__ __forceinline__ void store_lse(const KvAttn& A, int64_t t, int qh, float M, float L) {
  A.lse[t * A.q_heads + qh] = L == 0.0f ? -__builtin_inff() : (M + __builtin_amdgcn_logf(L)) * 0.693147180559945309f;
}

template <int E>
__device__ __forceinline__ void store_few(void* p, bool f32, int64_t off, const float (&x)[E]) {
  if constexpr (E == 2) {
    if (f32)
      *reinterpret_cast<float2*>(static_cast<float*>(p) + off) = make_float2(x[0], x[1]);
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p) + off) = pack_bf16(x[0], x[1]);
  } else {
    store_whole(p, f32, off, x);
  }
}

template <int FMT, int D, int NR, int kWaves, bool NT>
__global__ __launch_bounds__(64 * kWaves, waves_of(D, NR)) void kv_attn_kernel(KvAttn A) {
  using G = Geo<FMT, D>;
  constexpr int LD = D + 4;                            // a row in LDS: the lanes' rows meet different banks
  constexpr int kKeys = 32 * kWaves;                   // of a round of the waves
  constexpr int kUnit = kRows * NR;
  __shared__ float stats[2][kWaves][kRows];
  __shared__ f4_t part[kWaves][kRows * LD / 4];
  __shared__ int upto[kWaves][2][64];
  const int lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ek = G::NV ? entries(A.c.texp)[0] : 0, ev = G::NV ? entries(A.c.texp)[1] : 0;
  Cursor cur;
  cur.coarse = upto[wave][0];
  cur.fine = upto[wave][1];
  cur.unit_rows = kUnit;
  const Shares shares(cur.total(A), gridDim.x);
  int at = shares.first(blockIdx.x);
  const int stop = shares.first(blockIdx.x + 1);
  if (at >= stop) {
    if (A.left && threadIdx.x == 0) A.left[blockIdx.x] = Left{0, 0, 0, 0, 0};
    return;
  }

  // A share's part of a unit. Its queries and first keys are asked for before the
  // one before it is joined.
  struct Part {
    int64_t row0, pos0;
    int seq, head, r0, rows;
    int begin, last;           // keys
    bool all, goes_on;         // the whole unit; a unit that an earlier workgroup began
    int owner;                 // of the unit's last step
  };
  Rows<FMT, D> R[NR];
  Tile<FMT, D> T0, T1;
  struct Pages {
    int p[2];
  };
  Pages g0, g1;
  auto setup = [&](Part& P) {
    int from;
    P.seq = cur.seek(A, at, &from);
    const Span U = span_of(A, P.seq, kUnit);
    const int unit = (at - from) / U.steps, s0 = (at - from) % U.steps;
    const int s1 = stop - at < U.steps - s0 ? s0 + (stop - at) : U.steps;
    at += s1 - s0;
    P.row0 = U.row0;
    P.pos0 = U.pos0;
    P.head = unit / U.tiles;
    P.r0 = unit % U.tiles * kUnit;
    P.rows = U.rows - P.r0 < kUnit ? U.rows - P.r0 : kUnit;
    const int64_t begin = (int64_t)(first_key(A, U.pos0) & ~31) + (int64_t)s0 * A.step, end = begin + (int64_t)(s1 - s0) * A.step - 1;
    const int unit_last = limit(A, U.pos0 + (P.r0 + P.rows - 1) / A.group);
    P.begin = (int)begin;
    P.last = end < unit_last ? (int)end : unit_last;
    P.all = s1 - s0 == U.steps;
    P.goes_on = s0 > 0;
    P.owner = P.all ? 0 : shares.owner(at - s1 + U.steps - 1);
  };
  // The table's entries are asked for two rounds ahead.
  auto pages = [&](const Part& P, int key) {
    const Entries table = entries(A.b.table + (int64_t)P.seq * A.b.table_ld);
    Pages g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = key + 16 * h < P.last ? key + 16 * h : P.last;
      g.p[h] = table[(k > 0 ? k : 0) >> A.c.shift];
    }
    return g;
  };
  auto mapped = [&](const Pages& g, int h) { return (uint32_t)g.p[h] < (uint32_t)A.c.pages; };
  // Loads are never skipped, since the wait for a tile counts those of the next
  // one: beyond the last key, and where a page is not mapped, they read others.
  auto load = [&](const Part& P, int key, const Pages& g, Tile<FMT, D>& T) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      load_half<FMT, D, NT>(A.c, kv_slot(A.c, mapped(g, h) ? g.p[h] : 0, P.head, (key + 16 * h) & ((1 << A.c.shift) - 1)), T.k[h],
                        T.ks[h], T.v[h], T.vs[h]);
  };
  auto issue = [&](const Part& P) {
    const int key = P.begin + 32 * wave;
    g0 = pages(P, key);
    g1 = pages(P, key + kKeys);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = P.r0 + kRows * i + n;
      R[i].load(kRows * i + n < P.rows
                    ? A.q + (P.row0 + r / A.group) * A.ldq + (int64_t)(P.head * A.group + r % A.group) * D
                    : nullptr);
    }
    load(P, key, g0, T0);
  };

  Left left = {0, 0, 0, 0, 0};
  Part P;
  setup(P);
  issue(P);
  while (true) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = kRows * i + n;
      const int64_t pos = P.pos0 + (P.r0 + r) / A.group;
      R[i].start(A.scale, ek);
      R[i].last = r < P.rows ? limit(A, pos) : -1;
      R[i].first = first_key(A, pos);
    }
    // keys of any row of the unit, and of all
    const int64_t p0 = P.pos0 + P.r0 / A.group, p1 = P.pos0 + (P.r0 + P.rows - 1) / A.group;
    const int first = first_key(A, p0), every_first = first_key(A, p1), every_last = limit(A, p0), last = P.last;
    auto use = [&](int key, const Pages& g, Tile<FMT, D>& T) {
      // scores: s[i][h][j] is key 16 h + 4 c + j for row n of tile i
      f4_t s[NR][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < NR; ++i) s[i][h] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
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
            const int b = G::SB == 2 ? w / 2 : 0;      // block of the piece
            const u32x4_t k = decode_key<FMT>(T.k[h][l][w], h2_t{sc[b], sc[b]}, e);
#pragma unroll
            for (int i = 0; i < NR; ++i) s[i][h] = mfma<FMT>(k, R[i].q[l][w], s[i][h]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][h][j] *= R[i].factor;
      const bool whole = mapped(g, 0) & mapped(g, 1) & (key >= every_first) & (key + 31 <= every_last);
      if (!whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k0 = key + 16 * h + 4 * c, end = mapped(g, h) ? last : -1;
          uint32_t keep = 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
              s[i][h][j] = ((k0 + j >= R[i].first) & (k0 + j <= R[i].last) & (k0 + j <= end)) ? s[i][h][j] : -__builtin_inff();
            keep |= ((k0 + j >= first) & (k0 + j <= end)) ? 0xFFu << (8 * j) : 0u;
          }
          // values of places that no row sees may be anything: their scales are replaced
#pragma unroll
          for (int l = 0; l < G::VL; ++l) T.vs[h][l] &= keep;
        }
      }
      // The maximum may lag by 2^8: terms of up to 256 are as exact, and most tiles leave the output as it is.
      float top[NR];
      bool above = false;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        top[i] = kLowest;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) top[i] = fmaxf(top[i], s[i][h][j]);
        above |= top[i] > R[i].m + 8.0f;
      }
      if (__any(above)) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float m = fmaxf(row_max(top[i]), R[i].m), f = __builtin_amdgcn_exp2f(R[i].m - m);
          R[i].m = m;
          R[i].l *= f;
#pragma unroll
          for (int d = 0; d < G::DT; ++d) R[i].o[d] *= f;
        }
      }
      u32x4_t ph[NR], pl[NR];                          // fp16, or the two parts in bf16
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] = __builtin_amdgcn_exp2f(s[i][j / 4][j % 4] - R[i].m);
          R[i].l += p[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (G::NV) {
            ph[i][j] = bits(h2_t{(_Float16)p[2 * j], (_Float16)p[2 * j + 1]});
          } else {
            ph[i][j] = pack_bf16(p[2 * j], p[2 * j + 1]);
            pl[i][j] = pack_bf16(p[2 * j] - bf16_lo(ph[i][j]), p[2 * j + 1] - bf16_hi(ph[i][j]));
          }
        }
      }
#pragma unroll
      for (int l = 0; l < G::VL; ++l) {
        uint32_t v0[2 * G::VB][2], v1[2 * G::VB][2];
        decode_values<FMT, D>(T.v[0][l], T.vs[0][l], v0);
        decode_values<FMT, D>(T.v[1][l], T.vs[1][l], v1);
#pragma unroll
        for (int d = 0; d < 2 * G::VB; ++d) {
          const u32x4_t a = {v0[d][0], v0[d][1], v1[d][0], v1[d][1]};
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            f4_t& o = R[i].o[l * 2 * G::VB + d];
            o = mfma<FMT>(a, ph[i], o);
            if constexpr (!G::NV) o = mfma<FMT>(a, pl[i], o);
          }
        }
      }
    };

    int key = P.begin + 32 * wave;
    if (key <= last) {
      while (true) {
        load(P, key + kKeys, g1, T1);
        const Pages g2 = pages(P, key + 2 * kKeys);
        use(key, g0, T0);
        key += kKeys;
        if (key > last) break;
        load(P, key + kKeys, g2, T0);
        const Pages g3 = pages(P, key + 2 * kKeys);
        use(key, g1, T1);
        key += kKeys;
        if (key > last) break;
        g0 = g2;
        g1 = g3;
      }
    }
    const bool more = at < stop;
    Part N = P;
    if (more) {
      setup(N);
      issue(N);
    }

    // the waves' shares of the rows, joined, a tile at a time: the unit's output, or one of the workgroup's two slots
    float* slot = A.part + (2 * (int64_t)blockIdx.x + !P.goes_on) * slot_floats(D, kUnit);
    if (!P.all && !P.goes_on) left = Left{P.row0, P.rows, P.r0, P.head, P.owner};
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      if (kRows * i >= P.rows) break;
      const float l = row_sum(R[i].l);
      if (c == 0) {
        stats[0][wave][n] = R[i].m;
        stats[1][wave][n] = l;
      }
#pragma unroll
      for (int v = 0; v < G::VL; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j)                    // O^T's row 4 c + j in 2 VB tiles: dimensions in a row
#pragma unroll
          for (int d = 0; d < 2 * G::VB; d += 4)
            part[wave][(n * LD + v * 32 * G::VB + (4 * c + j) * 2 * G::VB + d) / 4] =
                f4_t{R[i].o[v * 2 * G::VB + d][j], R[i].o[v * 2 * G::VB + d + 1][j], R[i].o[v * 2 * G::VB + d + 2][j], R[i].o[v * 2 * G::VB + d + 3][j]};
      __syncthreads();
      constexpr int LR = 4 * kWaves;                   // lanes of a row
      constexpr int E = D / LR < 4 ? D / LR : 4;
      const int row = threadIdx.x / LR, d0 = threadIdx.x % LR * (D / LR);
      float M = kLowest, L = 0.0f, w[kWaves];
#pragma unroll
      for (int k = 0; k < kWaves; ++k) M = fmaxf(M, stats[0][k][row]);
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        w[k] = __builtin_amdgcn_exp2f(stats[0][k][row] - M);
        L += stats[1][k][row] * w[k];
      }
      const int ur = kRows * i + row;
      if (ur < P.rows) {
        const int rr = P.r0 + ur;
        const int64_t t = P.row0 + rr / A.group;
        const int qh = P.head * A.group + rr % A.group;
        const float inv = !P.all ? 1.0f : L == 0.0f ? 0.0f : ldexpf(1.0f / L, ev);
#pragma unroll
        for (int d = 0; d < D / LR; d += E) {
          float x[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            x[e] = 0.0f;
#pragma unroll
            for (int k = 0; k < kWaves; ++k) x[e] += reinterpret_cast<const float*>(part[k])[row * LD + d0 + d + e] * w[k];
            x[e] *= inv;
          }
          if (P.all)
            store_few(A.out, false, t * A.ldo + (int64_t)qh * D + d0 + d, x);
          else
            store_few(slot, true, 2 * kUnit + ur * D + d0 + d, x);
        }
        if (d0 == 0) {
          if (!P.all) {
            slot[ur] = M;
            slot[kUnit + ur] = L;
          } else if (A.lse) {
            store_lse(A, t, qh, M, L);
          }
        }
      }
      if (i + 1 < NR || more) __syncthreads();
    }
    if (!more) break;
    P = N;
  }
  if (A.left && threadIdx.x == 0) A.left[blockIdx.x] = left;
}

// A unit that several workgroups had a share of, joined: blockIdx.x is the one
// that has its first step, blockIdx.y the row. The parts are taken by several
// groups of lanes and added in a fixed order.
template <int D, int NR>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttn A, bool nv) {
  constexpr int LR = D / 4, SUBS = 256 / LR;           // lanes of a row, parts taken at once
  constexpr int kUnit = kRows * NR;
  __shared__ float sm[SUBS], sl[SUBS];
  __shared__ f4_t so[SUBS][LR];
  const int w0 = blockIdx.x, row = blockIdx.y;
  const Left U = A.left[w0];
  if (row >= U.rows) return;
  const int w1 = U.last;
  auto slot = [&](int w) { return A.part + (2 * (int64_t)w + (w == w0)) * slot_floats(D, kUnit); };
  const int sub = threadIdx.x / LR, d = threadIdx.x % LR * 4;
  float M = kLowest, L = 0.0f;
  f4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (w1 - w0 < SUBS) {
    if (w0 + sub <= w1) {
      const float* p = slot(w0 + sub);
      M = p[row];
      L = p[kUnit + row];
      x = *reinterpret_cast<const f4_t*>(p + 2 * kUnit + row * D + d);
    }
  } else {
    for (int w = w0 + sub; w <= w1; w += 4 * SUBS) {   // four parts in flight
      f4_t v[4];
      float m[4], l[4], top = M;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = w + u * SUBS <= w1;
        const float* p = slot(in ? w + u * SUBS : w);
        m[u] = in ? p[row] : kLowest;
        l[u] = in ? p[kUnit + row] : 0.0f;
        v[u] = *reinterpret_cast<const f4_t*>(p + 2 * kUnit + row * D + d);
        if (!in) v[u] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) top = fmaxf(top, m[u]);
      const float old = __builtin_amdgcn_exp2f(M - top);
      M = top;
      L *= old;
      x *= old;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = __builtin_amdgcn_exp2f(m[u] - M);
        L += l[u] * f;
        x += v[u] * f;
      }
    }
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
  if (A.lse && d == 0) store_lse(A, t, qh, M, L);
}

// Many rows a sequence: a workgroup has a unit of 64 NR rows, a wave 16 NR of
// them, and all keys of the unit. The waves decode 16 of 64 keys each into LDS, in
// the order of the products' operands, for all of them: a quarter of the decoding
// a wave, and one barrier for 64 keys, with two buffers.
template <int FMT, int D>
struct Half {                  // what a lane holds of 16 tokens
  using G = Geo<FMT, D>;
  uint32_t k[G::KL][G::KD], ks[G::KL];
  uint32_t v[G::VL][G::VB], vs[G::VL];
};

constexpr int prompt_tiles(int dim) { return dim == 256 ? 1 : 2; }      // NR
constexpr int prompt_halves(int dim) { return dim == 256 ? 2 : 4; }

template <int FMT, int D, int NR>
__global__ __launch_bounds__(64 * kWaves, D == 64 ? 3 : 2) void kv_prompt_kernel(KvAttn A) {
  using G = Geo<FMT, D>;
  constexpr int KH = prompt_halves(D);                 // halves of 16 keys at a time: a wave's both, or keys or values
  constexpr int kUnit = kRows * NR * kWaves, kKeys = 16 * KH, KC = G::KL * G::KD;
  __shared__ u32x4_t keys[2][KH][KC][64];              // [half of 16 keys][32 dimensions][lane]
  __shared__ u32x2_t vals[2][KH / 2][G::DT][64][2];    // [32 keys][tile of 16 dimensions][lane][half]
  const int lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // heads first: a head's units meet in one XCD's cache; of a sequence's units those with the most keys
  // first; every other round of the CUs goes the other way, so that a CU gets long and short ones
  const int head = blockIdx.x % A.c.heads, round = A.c.heads < 256 ? 256 / A.c.heads : 1;
  int place = blockIdx.x / A.c.heads;
  if (place / round % 2 == 1 && (place / round + 1) * round * A.c.heads <= (int)gridDim.x) place = (place / round * 2 + 1) * round - 1 - place;
  auto start = [&](int i) { return (int64_t)A.b.cu[i] * A.group / kUnit + i; };
  const int seq = A.b.cu ? kv_find(A.b.seqs, place, start) : place / ((A.group + kUnit - 1) / kUnit);
  if (seq < 0 || seq >= A.b.seqs) return;
  const Span U = span_of(A, seq, kUnit);
  const int64_t base = A.b.cu ? (int64_t)entries(A.b.cu)[seq] * A.group / kUnit + seq : (int64_t)seq * U.tiles;
  const int64_t tile = U.tiles - 1 - (place - base);
  if (tile < 0 || tile >= U.tiles || U.rows <= A.few) return;
  const int ek = G::NV ? entries(A.c.texp)[0] : 0, ev = G::NV ? entries(A.c.texp)[1] : 0;
  const int r0 = (int)tile * kUnit, w0 = r0 + wave * kRows * NR;
  const int rows = U.rows - r0 < kUnit ? U.rows - r0 : kUnit, wrows = U.rows - w0;
  Rows<FMT, D> R[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = w0 + kRows * i + n, tok = r / A.group;
    const bool mine = kRows * i + n < wrows;
    R[i].load(mine ? A.q + (U.row0 + tok) * A.ldq + (int64_t)(head * A.group + r % A.group) * D : nullptr);
    R[i].start(A.scale, ek);
    R[i].factor = fmaxf(R[i].factor, 1.0e-37f);        // times -inf is -inf
    R[i].last = mine ? limit(A, U.pos0 + tok) : -1;
    R[i].first = first_key(A, U.pos0 + tok);
  }
  // keys of any row of the unit; of any and of all rows of the wave
  const int first = first_key(A, U.pos0 + r0 / A.group), last = limit(A, U.pos0 + (r0 + rows - 1) / A.group);
  const int wlast = wrows > 0 ? limit(A, U.pos0 + (w0 + (wrows < kRows * NR ? wrows : kRows * NR) - 1) / A.group) : -1;
  const int wfirst = first_key(A, U.pos0 + w0 / A.group);
  const int every_first = first_key(A, U.pos0 + (w0 + kRows * NR - 1) / A.group), every_last = limit(A, U.pos0 + w0 / A.group);
  const Entries table = entries(A.b.table + (int64_t)seq * A.b.table_ld);

  struct Pages {
    int p[KH];
  };
  auto pages = [&](int key) {
    Pages g;
#pragma unroll
    for (int h = 0; h < KH; ++h) g.p[h] = table[(key + 16 * h < last ? key + 16 * h : last) >> A.c.shift];
    return g;
  };
  auto mapped = [&](int p) { return (uint32_t)p < (uint32_t)A.c.pages; };
  const int half = wave % KH;                          // what the wave decodes
  const bool do_keys = KH == kWaves || wave < KH, do_values = KH == kWaves || wave >= KH;
  auto entry = [&](int key) { return table[(key + 16 * half < last ? key + 16 * half : last) >> A.c.shift]; };
  auto load = [&](int key, int p, Half<FMT, D>& T) {
    load_half<FMT, D>(A.c, kv_slot(A.c, mapped(p) ? p : 0, head, (key + 16 * half) & ((1 << A.c.shift) - 1)), T.k, T.ks, T.v, T.vs);
  };
  auto decode = [&](int key, int buf, int p, Half<FMT, D>& T) {
    const int k0 = key + 16 * half, end = mapped(p) ? last : -1;
    if (k0 < first || k0 + 15 > end) {
      // values of places that no row sees may be anything: their scales are replaced
    uint32_t keep = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) keep |= ((k0 + 4 * c + j >= first) & (k0 + 4 * c + j <= end)) ? 0xFFu << (8 * j) : 0u;
#pragma unroll
      for (int l = 0; l < G::VL; ++l) T.vs[l] &= keep;
    }
    if (do_keys) {
#pragma unroll
    for (int l = 0; l < G::KL; ++l) {
      h2_t sc = {};
      float e = 0.0f;
      if constexpr (G::NV)
        sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(T.ks[l], 1.0f, false);
      else
        e = e8m0_val(T.ks[l]);
#pragma unroll
      for (int w = 0; w < G::KD; ++w) {
        const int b = G::SB == 2 ? w / 2 : 0;
        keys[buf][half][l * G::KD + w][lane] = decode_key<FMT>(T.k[l][w], h2_t{sc[b], sc[b]}, e);
      }
    }
    }
    if (do_values) {
#pragma unroll
    for (int l = 0; l < G::VL; ++l) {
      uint32_t v[2 * G::VB][2];
      decode_values<FMT, D>(T.v[l], T.vs[l], v);
#pragma unroll
      for (int d = 0; d < 2 * G::VB; ++d) vals[buf][half / 2][l * 2 * G::VB + d][lane][half % 2] = u32x2_t{v[d][0], v[d][1]};
    }
    }
  };
  auto use = [&](int key, int buf, const Pages& g) {
    f4_t s[NR][KH];
    if constexpr (D == 128) __builtin_amdgcn_s_setprio(1);   // over the other workgroup's softmax (187 -> 183 us)
#pragma unroll
    for (int h = 0; h < KH; ++h) {
#pragma unroll
      for (int i = 0; i < NR; ++i) s[i][h] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < KC; ++w) {
        const u32x4_t k = keys[buf][h][w][lane];
#pragma unroll
        for (int i = 0; i < NR; ++i) s[i][h] = mfma<FMT>(k, R[i].q[w / G::KD][w % G::KD], s[i][h]);
      }
    }
    if constexpr (D == 128) __builtin_amdgcn_s_setprio(0);
    bool whole = (key >= every_first) & (key + kKeys - 1 <= every_last);
#pragma unroll
    for (int h = 0; h < KH; ++h) whole &= mapped(g.p[h]);
    if (!whole) {
#pragma unroll
      for (int h = 0; h < KH; ++h) {
        const int k0 = key + 16 * h + 4 * c, end = mapped(g.p[h]) ? last : -1;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < NR; ++i)
            s[i][h][j] = ((k0 + j >= R[i].first) & (k0 + j <= R[i].last) & (k0 + j <= end)) ? s[i][h][j] : -__builtin_inff();
      }
    }
    float top[NR];
    bool above = false;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      top[i] = kLowest;
#pragma unroll
      for (int h = 0; h < KH; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) top[i] = fmaxf(top[i], s[i][h][j]);
      top[i] *= R[i].factor;
      above |= top[i] > R[i].m + 8.0f;
    }
    if (__any(above)) {
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float m = fmaxf(row_max(top[i]), R[i].m), f = __builtin_amdgcn_exp2f(R[i].m - m);
        R[i].m = m;
        R[i].l *= f;
#pragma unroll
        for (int d = 0; d < G::DT; ++d) R[i].o[d] *= f;
      }
    }
#pragma unroll
    for (int pr = 0; pr < KH / 2; ++pr) {
      u32x4_t ph[NR], pl[NR];                          // fp16, or the two parts in bf16
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][2 * pr + j / 4][j % 4], R[i].factor, -R[i].m));
          R[i].l += p[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (G::NV) {
            ph[i][j] = bits(h2_t{(_Float16)p[2 * j], (_Float16)p[2 * j + 1]});
          } else {
            ph[i][j] = pack_bf16(p[2 * j], p[2 * j + 1]);
            pl[i][j] = pack_bf16(p[2 * j] - bf16_lo(ph[i][j]), p[2 * j + 1] - bf16_hi(ph[i][j]));
          }
        }
      }
      if constexpr (D == 128) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int d = 0; d < G::DT; ++d) {
        const u32x4_t a = *reinterpret_cast<const u32x4_t*>(vals[buf][pr][d][lane]);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          R[i].o[d] = mfma<FMT>(a, ph[i], R[i].o[d]);
          if constexpr (!G::NV) R[i].o[d] = mfma<FMT>(a, pl[i], R[i].o[d]);
        }
      }
      if constexpr (D == 128) __builtin_amdgcn_s_setprio(0);
    }
  };

  // Codes are loaded two tiles ahead of their decoding, and decoded one ahead of
  // their use, whether or not there are keys left (see kv_attn_kernel). The
  // table's entries are asked for before a barrier, which waits for them.
  int key = first & ~15;
  if (key <= last) {
    Half<FMT, D> T0, T1;
    int e0 = entry(key), e1 = entry(key + kKeys), e2 = entry(key + 2 * kKeys), e3 = entry(key + 3 * kKeys);
    Pages g = pages(key);
    load(key, e0, T0);
    load(key + kKeys, e1, T1);
    decode(key, 0, e0, T0);
    load(key + 2 * kKeys, e2, T0);
    __syncthreads();
    auto tile = [&](int buf, Half<FMT, D>& T) {
      decode(key + kKeys, buf ^ 1, e1, T);
      load(key + 3 * kKeys, e3, T);
      if (key <= wlast && key + kKeys > wfirst) use(key, buf, g);
      key += kKeys;
      e1 = e2;
      e2 = e3;
      e3 = entry(key + 3 * kKeys);
      g = pages(key);
      __syncthreads();
    };
    while (true) {
      tile(0, T1);
      if (key > last) break;
      tile(1, T0);
      if (key > last) break;
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const float L = row_sum(R[i].l), inv = L == 0.0f ? 0.0f : ldexpf(1.0f / L, ev);
    if (kRows * i + n >= wrows) continue;
    const int r = w0 + kRows * i + n;
    const int64_t t = U.row0 + r / A.group;
    const int qh = head * A.group + r % A.group;
#pragma unroll
    for (int l = 0; l < G::VL; ++l)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[2 * G::VB];
#pragma unroll
        for (int d = 0; d < 2 * G::VB; ++d) x[d] = R[i].o[l * 2 * G::VB + d][j] * inv;
        store_whole(A.out, false, t * A.ldo + (int64_t)qh * D + l * 32 * G::VB + (4 * c + j) * 2 * G::VB, x);
      }
    if (A.lse && c == 0) store_lse(A, t, qh, R[i].m, L);
  }
}

// Keys up to which a workgroup takes a unit as a whole: the second launch costs
// as much as five rounds of eight waves.
constexpr int kShort = 1280;
// Bytes of a cache from which it is read past the last-level cache.
constexpr int64_t kStream = (int64_t)128 << 20;

}  // namespace

int64_t kv_attn_tiles(int64_t tokens, int64_t seqs, int64_t group) { return tokens * group / kRows + seqs; }

size_t kv_attn_slots(int dim) {
  size_t most = 0;
  for (int t = 1; t <= most_tiles(dim); ++t) {
    const size_t n = (size_t)workers_of(dim, t) * (2 * slot_floats(dim, kRows * t) * sizeof(float) + sizeof(Left));
    most = n > most ? n : most;
  }
  return most;
}

hipError_t launch_kv_attn(int format, int dim, KvAttn a, hipStream_t s) {
  const bool nv = format == SNIP_NVFP4;
  const int64_t rows = a.tokens * a.group / a.b.seqs;    // of a sequence, on average
  const int unit = kRows * kWaves * prompt_tiles(dim);
  const int64_t places = a.b.cu ? a.tokens * a.group / unit + a.b.seqs : (int64_t)a.b.seqs * ((a.group + unit - 1) / unit);
  const bool prompt = rows >= 64 && a.tokens * a.group / unit * a.c.heads >= 256 && places * a.c.heads < (1 << 24);
  a.split = prompt && a.b.seqs > 1;
  a.few = a.split ? 64 : 0;
  // Short tables: a workgroup a unit and no second launch.
  const bool whole = a.b.max_len <= kShort && !prompt;
  const double tiles = (double)kv_attn_tiles(a.tokens, a.b.seqs, a.group) * a.c.heads;
  const bool wide = whole && tiles <= 512.0;
  const bool two = dim != 256 && rows > kRows && !wide;
  // steps are counted in 31 bits, whatever the lengths that the tables allow
  a.step = 32 * kWaves;
  while (a.step < a.b.max_len && (whole || tiles * ((double)a.b.max_len / a.step + 1.0) >= 2147483647.0)) a.step *= 2;
  const int blk = nv ? 16 : 32;
  const bool nt = !whole && ((int64_t)a.c.pages * a.c.heads << a.c.shift) * (dim + 2 * dim / blk) >= kStream;

  auto go = [&](auto f, auto d, auto t) {
    constexpr int FMT = decltype(f)::value, D = decltype(d)::value, NR = decltype(t)::value, W = workers_of(D, NR);
    if (prompt) {
      kv_prompt_kernel<FMT, D, prompt_tiles(D)><<<(unsigned)(places * a.c.heads), 64 * kWaves, 0, s>>>(a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess || !a.split) return e;
    }
    if (whole) {
      const int64_t most = (a.b.cu ? a.tokens * a.group / (kRows * NR) + a.b.seqs
                                   : (int64_t)a.b.seqs * ((a.group + kRows * NR - 1) / (kRows * NR))) * a.c.heads;
      const unsigned grid = (unsigned)(most < (1 << 20) ? most : 1 << 20);
      a.left = nullptr;
      if constexpr (NR == 1) {
        if (wide) {
          kv_attn_kernel<FMT, D, 1, 8, false><<<grid, 64 * 8, 0, s>>>(a);
          return hipGetLastError();
        }
      }
      kv_attn_kernel<FMT, D, NR, kWaves, false><<<grid, 64 * kWaves, 0, s>>>(a);
      return hipGetLastError();
    }
    a.left = reinterpret_cast<Left*>(a.part + (size_t)W * 2 * slot_floats(D, kRows * NR));
    if (nt)
      kv_attn_kernel<FMT, D, NR, kWaves, true><<<W, 64 * kWaves, 0, s>>>(a);
    else
      kv_attn_kernel<FMT, D, NR, kWaves, false><<<W, 64 * kWaves, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int most = !a.b.cu && a.group < kRows * NR ? a.group : kRows * NR;   // rows of a unit
    kv_join_kernel<D, NR><<<dim3(W - 1, most), 256, 0, s>>>(a, nv);
    return hipGetLastError();
  };
  auto of = [&](auto f, auto d) {
    if constexpr (most_tiles(decltype(d)::value) > 1)
      if (two) return go(f, d, std::integral_constant<int, 2>{});
    return go(f, d, std::integral_constant<int, 1>{});
  };
  auto at = [&](auto f) {
    return dim == 64    ? of(f, std::integral_constant<int, 64>{})
           : dim == 128 ? of(f, std::integral_constant<int, 128>{})
                        : of(f, std::integral_constant<int, 256>{});
  };
  return nv ? at(std::integral_constant<int, SNIP_NVFP4>{}) : at(std::integral_constant<int, SNIP_MXFP4>{});
}

}  // namespace snip
