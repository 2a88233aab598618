// Attention over a 4-bit key/value cache for sequences with many new tokens,
// gfx950 (mathematics and operand layouts: kv_tile.h).
//
// Many rows a sequence: a workgroup has a unit of 128 rows (64 with heads of 256)
// and all its keys; a wave has 16 NR of the rows. The keys and values are decoded
// into LDS once for all waves, in the order of the products' operands: a wave
// decodes the keys or the values of 16 tokens, so that W waves share 8 W tokens
// and one barrier, with two buffers. Both products' operands are then read from
// LDS, which binds: a read of 16 bytes a lane feeds NR products (MXFP4's values
// two each). W = 4 with NR = 2 reads half as much, W = 8 with NR = 1 has twice
// the waves for a grid that leaves CUs with few. Measured, us, W = 4 and W = 8,
// one NVFP4 sequence:
//     tokens = keys, 32 heads of 128    1024: 41, 32   3200: 116, 103   4096: 157, 160   8192: 540, 568
//     the same, 32 heads of 64          1024: 25, 20   3200: 72, 68     4096: 93, 103    8192: 328, 352
//     2048 after 4096, 32 heads of 128  210, 184
// 4096 tokens are 1024 workgroups there, four to a CU: below that, eight waves.
// Long prompts with heads of 128 reach 1093 TFLOP/s (16384 tokens), of 64 850: 8
// vector instructions to a product, against 4.8, mostly the softmax's.
// Heads of 256 have no LDS for eight waves of 64 rows; with units of 128 rows six
// sequences of 69 to 333 new tokens took 86 us for 69.
#include "kv_tile.h"

namespace snip {

namespace {

// What a lane holds of 16 tokens' keys, or of their values.
template <int FMT, int D>
struct Half {
  using G = Geo<FMT, D>;
  static_assert(G::KL == G::VL && G::KD == G::VB && G::PB == 4 * G::VB, "");
  uint32_t w[G::KL][G::KD], sc[G::KL];
};

template <int FMT, int D, int W>
__global__ __launch_bounds__(64 * W, D > 64 ? 2 : W == 4 ? 3 : 4) void kv_prompt_kernel(KvAttn A) {
  using G = Geo<FMT, D>;
  constexpr int kUnit = kv_prompt_rows(D), NR = kUnit / (kRows * W);
  constexpr int KH = W / 2;                            // halves of 16 keys at a time
  constexpr int kKeys = 16 * KH, KC = G::KL * G::KD;
  __shared__ u32x4_t keys[2][KH][KC][64];              // [half of 16 keys][32 dimensions][lane]
  __shared__ alignas(16) u32x2_t vals[2][KH / 2][G::DT][64][2];    // [32 keys][tile of 16 dimensions][lane][half]
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
  if (tile < 0 || tile >= U.tiles || !prompt_rows(A, U)) return;
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
    R[i].factor = fmaxf(R[i].factor, 1.0e-45f);        // the smallest above 0: times -inf is -inf
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
  // What the wave decodes, and where a lane's share of it lies: codes in pieces of
  // 16 bytes (8), scales in a word, from its bit `down` on.
  const int half = wave % KH;
  const bool do_keys = wave < KH;
  uint32_t code_at[G::KL], scale_at[G::KL], down[G::KL];
#pragma unroll
  for (int l = 0; l < G::KL; ++l) {
    const int ks = G::SB == 2 ? (64 * l + lane) * 2 : 2 * G::PB < G::BLK ? c / 2 * 16 + n : 64 * l + lane;
    code_at[l] = do_keys ? (64 * l + lane) * G::PB : c * 2 * D + (16 * l + n) * 4 * G::VB;
    scale_at[l] = do_keys ? ks & ~3 : c * 4 * (D / G::BLK) + (16 * l + n) * 2 * G::VB / G::BLK * 4;
    down[l] = do_keys ? 8 * (ks & 3) : 0;
  }
  const uint8_t* const codes = do_keys ? A.c.kc : A.c.vc;
  const uint8_t* const scales = do_keys ? A.c.ks : A.c.vs;
  auto entry = [&](int key) { return table[(key + 16 * half < last ? key + 16 * half : last) >> A.c.shift]; };
  auto load = [&](int key, int p, Half<FMT, D>& T) {
    const int64_t slot = kv_slot(A.c, mapped(p) ? p : 0, head, (key + 16 * half) & ((1 << A.c.shift) - 1));
#pragma unroll
    for (int l = 0; l < G::KL; ++l) {
      load_words<false>(codes + slot * (D / 2) + code_at[l], T.w[l]);
      T.sc[l] = *reinterpret_cast<const uint32_t*>(scales + slot * (D / G::BLK) + scale_at[l]);
    }
  };
  auto decode = [&](int key, int buf, int p, Half<FMT, D>& T) {
    if (do_keys) {
#pragma unroll
      for (int l = 0; l < G::KL; ++l) {
        const uint32_t b = T.sc[l] >> down[l];
        h2_t sc = {};
        float e = 0.0f;
        if constexpr (G::NV)
          sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
        else
          e = e8m0_val(b & 0xFFu);
#pragma unroll
        for (int w = 0; w < G::KD; ++w) {
          const int i = G::SB == 2 ? w / 2 : 0;        // block of the piece
          keys[buf][half][l * G::KD + w][lane] = decode_key<FMT>(T.w[l][w], h2_t{sc[i], sc[i]}, e);
        }
      }
      return;
    }
    const int k0 = key + 16 * half, end = mapped(p) ? last : -1;
    if (k0 < first || k0 + 15 > end) {
      // values of places that no row sees may be anything: their scales are replaced
      uint32_t keep = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) keep |= ((k0 + 4 * c + j >= first) & (k0 + 4 * c + j <= end)) ? 0xFFu << (8 * j) : 0u;
#pragma unroll
      for (int l = 0; l < G::VL; ++l) T.sc[l] &= keep;
    }
#pragma unroll
    for (int l = 0; l < G::VL; ++l) {
      uint32_t v[2 * G::VB][2];
      decode_values<FMT, D>(T.w[l], T.sc[l], v);
#pragma unroll
      for (int d = 0; d < 2 * G::VB; ++d) vals[buf][half / 2][l * 2 * G::VB + d][lane][half % 2] = u32x2_t{v[d][0], v[d][1]};
    }
  };
  auto use = [&](int key, int buf, const Pages& g) {
    f4_t s[NR][KH];
    if constexpr (D == 128) __builtin_amdgcn_s_setprio(1);   // over the other workgroup's softmax (16384 tokens: 2026 -> 1985 us; 7% more with heads of 64)
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
      above |= top[i] > R[i].m + (kLag + kLift<FMT>);
    }
    if (__any(above)) {
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float m = fmaxf(row_max(top[i]) - kLift<FMT>, R[i].m), f = __builtin_amdgcn_exp2f(R[i].m - m);
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
    const float L = row_sum(R[i].l), inv = L == 0.0f ? 0.0f : 1.0f / L;
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
        for (int d = 0; d < 2 * G::VB; ++d) x[d] = output<FMT>(R[i].o[l * 2 * G::VB + d][j], inv, ev);
        store_whole(A.out, false, t * A.ldo + (int64_t)qh * D + l * 32 * G::VB + (4 * c + j) * 2 * G::VB, x);
      }
    if (A.lse && c == 0) store_lse(A, t, qh, R[i].m, L);
  }
}

}  // namespace

hipError_t launch_kv_prompt(int format, int dim, const KvPlan& p, const KvAttn& a, hipStream_t s) {
  auto go = [&](auto f, auto d) {
    constexpr int F = decltype(f)::value, D = decltype(d)::value;
    if constexpr (D < 256) {
      if (p.prompt_waves == 8) {
        kv_prompt_kernel<F, D, 8><<<p.prompt_wg, 64 * 8, 0, s>>>(a);
        return hipGetLastError();
      }
    }
    kv_prompt_kernel<F, D, 4><<<p.prompt_wg, 64 * 4, 0, s>>>(a);
    return hipGetLastError();
  };
  return kv_dispatch(format, dim, go);
}

}  // namespace snip
