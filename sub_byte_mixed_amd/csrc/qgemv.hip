// y[M][N] = x[M][K] . dequant(w)[N][K]^T for 1..16 tokens, gfx950.
//
//   y[m][n] = 2^e sum_b s[n][b] sum_{k in block b} c[n][k] x[m][k]
//
// Bound by the weights' bytes (0.53 to 1 byte each), read once; at a few MB by
// latency. Both forms below take the codes in 1 KB loads that run ahead of
// their use and multiply in bf16 with fp32 sums; codes are exact in bf16.
//  - dot: a wave has a row and the whole K; v_dot2_f32_bf16 on the
//    decoded pairs, the block scale on the block's sum. 36 VALU operations per
//    KB of codes and token, so it is for one or two tokens.
//  - MFMA: tiles of 16 rows x 16 tokens, the waves of a workgroup share K;
//    scales are applied as the codes are decoded (64 VALU operations per KB of
//    NVFP4, 16 of MXFP4, for all tokens).
// NVFP4, one token, dot / MFMA: 2048 x 2048 2.9 / 4.1 us, 4096 x 11008 7.2 /
// 8.5, 28672 x 8192 23.4 / 28.5 (5.6 TB/s; of 132 MB, a bare read takes 21.3).
// Times here and below: launches of a captured graph, one after the other, over
// weights that exceed the last-level cache.
#include "row_common.h"

namespace snip {

// How a format's weights are stored. SC: 0 none, 1 E4M3, 2 E8M0, 3 bf16.
template <int FMT>
struct WFmt {
  static constexpr bool FP8 = FMT == SNIP_FP8_E4M3;
  static constexpr int BLK = FMT == SNIP_MXFP4 || FMT == SNIP_FP4_E4M3_B32 || FMT == SNIP_FP4_BF16_B32 ? 32 : 16;
  static constexpr int SC = FP8 ? 0
                            : FMT == SNIP_NVFP4 || FMT == SNIP_FP4_E4M3_B32     ? 1
                            : FMT == SNIP_MXFP4 || FMT == SNIP_FP4_E8M0_B16     ? 2
                                                                                : 3;
  static constexpr int PER = FP8 ? 16 : 32;            // weights of one 16-byte load
  static constexpr int NB = FP8 ? 1 : PER / BLK;       // blocks among them
};

// Scale bytes of 32 weights.
template <int FMT>
constexpr int scale_unit() {
  using W = WFmt<FMT>;
  return W::SC == 0 ? 0 : (32 / W::BLK) * (W::SC == 3 ? 2 : 1);
}

__device__ __forceinline__ float scale_val(int sc, uint32_t raw, int i) {
  if (sc == 3) return __uint_as_float((raw >> (16 * i)) << 16);
  if (sc == 1) return i == 0 ? __builtin_amdgcn_cvt_f32_fp8((int)raw, 0) : __builtin_amdgcn_cvt_f32_fp8((int)raw, 1);
  const uint32_t b = (raw >> (8 * i)) & 0xFFu;
  // E8M0: 2^(b - 127); 0 is the subnormal 2^-127, 255 is NaN
  return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23);
}

// Pair `j` (weights 2j, 2j + 1) of a code word.
template <bool FP8>
__device__ __forceinline__ bf16x2_t decode_pair(uint32_t w, int j) {
  if constexpr (FP8) {
    return j == 0 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)
                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
  } else {
    switch (j) {
      case 0: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0);
      case 1: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1);
      case 2: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2);
      default: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3);
    }
  }
}

__device__ __forceinline__ void store_y(const Gemv& A, int64_t m, int64_t n, float v) {
  const int64_t i = m * A.ldy + n;
  if (A.y_type == SNIPOP_F32)
    static_cast<float*>(A.y)[i] = v;
  else
    static_cast<uint16_t*>(A.y)[i] = (uint16_t)pack_bf16(v, 0.0f);
}

// Buffer descriptor over `bytes` of p: a load whose offset lies beyond them
// returns zero, which stands in for rows and columns outside the operands.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(bytes > 0 ? bytes : 0), 0x00027000);
}
constexpr uint32_t kOutside = 0x80000000u;             // beyond every descriptor

// ------------------------------------------------------------ dot form
constexpr int kRowWaves = 8;
constexpr int kRowSlab = 32768;                        // the tokens' values held in LDS (64 KB)

// MT tokens (group blockIdx.y), a row a wave. A wave's load is 1 KB of the row;
// the tokens' values of the same chunk come from LDS, in pieces of 8 swizzled
// so that the lanes' 64-byte strides meet no bank twice. The next chunk is
// loaded before the present one is used; beyond K the descriptors give zeros.
// WALK: the tokens fit in one slab, and a wave goes on to the row `stride`
// further, its loads running on from row to row.
template <int FMT, int MT, bool WALK>
__global__ __launch_bounds__(64 * kRowWaves) void qgemv_row_kernel(Gemv A, int64_t stride) {
  using W = WFmt<FMT>;
  constexpr int NP = W::PER / 8;                       // pieces of a chunk
  constexpr int SB = W::SC == 0 ? 0 : W::NB * (W::SC == 3 ? 2 : 1);   // scale bytes of a chunk
  constexpr int SLAB = kRowSlab / MT;
  extern __shared__ u32x4_t smem[];                    // [MT][pieces of a slab]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t n = (int64_t)blockIdx.x * kRowWaves + wave;
  const int m0 = blockIdx.y * MT;
  const int K = (int)A.K, nch = K / W::PER;
  const int64_t crow = W::FP8 ? K : K / 2, srow = (int64_t)SB * nch;
  __amdgpu_buffer_rsrc_t cb, sb;
  auto turn_to = [&](int64_t row) {
    const bool in = row < A.N;
    cb = buffer_of(A.codes + (in ? row : 0) * crow, in ? crow : 0);
    if constexpr (SB > 0) sb = buffer_of(A.scales + (in ? row : 0) * srow, in ? srow : 0);
  };
  struct Chunk {
    u32x4_t w;
    uint32_t sc;
  };
  auto load = [&](Chunk& d, int c) {
    d.w = __builtin_amdgcn_raw_buffer_load_b128(cb, 16 * c, 0, 2);
    d.sc = 0u;
    if constexpr (SB == 1) d.sc = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(sb, c, 0, 0);
    if constexpr (SB == 2) d.sc = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(sb, 2 * c, 0, 0);
    if constexpr (SB == 4) d.sc = __builtin_amdgcn_raw_buffer_load_b32(sb, 4 * c, 0, 0);
  };
  // the tokens' values k0 .. k0 + end into LDS, filled up with zeros
  auto stage = [&](int k0, int end, int pieces) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const u32x4_t* x = reinterpret_cast<const u32x4_t*>(A.x + (m0 + m < A.M ? m0 + m : 0) * A.ldx + k0);
      for (int i = threadIdx.x; i < pieces; i += 64 * kRowWaves) {
        const int c = i / NP, j = i % NP;
        smem[m * pieces + c * NP + (j ^ (c / (16 / NP) % NP))] = 8 * i < end ? x[i] : u32x4_t{0u, 0u, 0u, 0u};
      }
    }
  };
  float acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = 0.0f;
  auto use = [&](const Chunk& d, int c, int pieces) {  // chunk c of the slab
    u32x4_t xp[MT][NP];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NP; ++j) xp[m][j] = smem[m * pieces + c * NP + (j ^ (c / (16 / NP) % NP))];
    float part[W::NB][MT];
#pragma unroll
    for (int b = 0; b < W::NB; ++b)
#pragma unroll
      for (int m = 0; m < MT; ++m) part[b][m] = 0.0f;
#pragma unroll
    for (int pair = 0; pair < W::PER / 2; ++pair) {
      constexpr int per = W::FP8 ? 2 : 4;
      const bf16x2_t v = decode_pair<W::FP8>(d.w[pair / per], pair % per);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float& p = part[pair * 2 * W::NB / W::PER][m];
        p = __builtin_amdgcn_fdot2_f32_bf16(v, __builtin_bit_cast(bf16x2_t, (uint32_t)xp[m][pair / 4][pair % 4]), p,
                                            false);
      }
    }
#pragma unroll
    for (int b = 0; b < W::NB; ++b) {
      const float f = W::SC == 0 ? 1.0f : scale_val(W::SC, d.sc, b);
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m] = W::SC == 0 ? acc[m] + part[b][m] : fmaf(part[b][m], f, acc[m]);
    }
  };
  auto finish = [&] {
    const int e = A.texp ? *A.texp : 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float v = wave_sum_f(acc[m]);
      if (lane == 0 && n < A.N && m0 + m < A.M) store_y(A, m0 + m, n, ldexpf(v, e));
      acc[m] = 0.0f;
    }
  };

  turn_to(n);
  Chunk a, b;
  load(a, lane);
  if constexpr (WALK) {
    const int steps = (nch + 63) / 64;                 // of 64 chunks, the last one filled up with zeros
    const int pieces = steps * 64 * NP;
    stage(0, K, pieces);
    __syncthreads();
    int s = 0;
    // by turns into a and b, so that no load is waited for to be copied;
    // true where the wave's last row is done
    auto step = [&](const Chunk& d, Chunk& ahead) {
      const bool turn = s + 1 == steps;
      if (turn) turn_to(n + stride);
      load(ahead, turn ? lane : 64 * (s + 1) + lane);
      use(d, 64 * s + lane, pieces);
      ++s;
      if (!turn) return false;
      finish();
      s = 0;
      n += stride;
      return n >= A.N;
    };
    while (!step(a, b) && !step(b, a)) {
    }
  } else {
    for (int k0 = 0; k0 < K; k0 += SLAB) {
      const int end = K - k0 < SLAB ? K - k0 : SLAB;
      const int steps = (end / W::PER + 63) / 64, pieces = steps * 64 * NP;
      if (k0) __syncthreads();
      stage(k0, end, pieces);
      __syncthreads();
      for (int s = 0; s < steps; ++s) {
        b = a;
        load(a, k0 / W::PER + 64 * (s + 1) + lane);
        use(b, 64 * s + lane, pieces);
      }
    }
    finish();
  }
}

// ------------------------------------------------------------ MFMA form
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// 8 weights (one code word of E2M1, two of E4M3) with their block scale ->
// 8 bf16. E4M3 codes, and E2M1 times an E4M3 or E8M0 scale (6 and 2
// significant bits), are exact in bf16. E2M1 times a bf16 scale has up to 9
// bits: it is the exact sum of `hi` and `lo`. Scales for which that does not
// hold (beyond_bf16) do not come here.
template <int FMT>
__device__ __forceinline__ void decode8(const u32x4_t& w, int i, float s, bf16x8_t& hi, bf16x8_t& lo) {
  using W = WFmt<FMT>;
  u32x4_t h, l;
  if constexpr (W::FP8) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = __builtin_bit_cast(uint32_t, decode_pair<true>(w[2 * i + (j >> 1)], j & 1));
  } else if constexpr (W::SC == 2) {
    h[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 0));
    h[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 1));
    h[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 2));
    h[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 3));
  } else {
    float q[8];
    fp4x8_dec(w[i], q);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = q[2 * j] * s, b = q[2 * j + 1] * s;
      h[j] = pack_bf16(a, b);
      if constexpr (W::SC == 3) l[j] = pack_bf16(a - bf16_lo(h[j]), b - bf16_hi(h[j]));
    }
  }
  hi = __builtin_bit_cast(bf16x8_t, h);
  if constexpr (W::SC == 3) lo = __builtin_bit_cast(bf16x8_t, l);
}

// Nonzero at 0x80808080 (E8M0) or 0x80008000 (bf16) where a scale of the word
// has no exact product with every code: E8M0 from 2^126 on, where 4 times it
// leaves bf16 (and NaN); bf16 from 2^125 on, and below 2^-125, where the last
// of the 9 bits does. A scale of 0 (a block of zeros) is none of them. 1 and 3
// operations a scale, once a workgroup.
template <int SC>
__device__ __forceinline__ uint32_t beyond_bf16(uint32_t w) {
  if constexpr (SC == 2) return ~(w + 0x03030303u) & w;      // a byte of 253 or more
  const uint32_t v = w & 0x7FFF7FFFu;
  return (v + 0x02000200u) | (~(v + 0x7F007F00u) & (v + 0x7FFF7FFFu));
}
template <int SC>
constexpr uint32_t beyond_mask() {
  return SC == 2 ? 0x80808080u : 0x80008000u;
}

// The tile of 16 RT rows from n0 on without that product, as the dot form: a
// row and token a wave, sums of codes times tokens and the scale on them. For
// tiles with a scale beyond_bf16: no quantizer writes one for finite values,
// unless they are below 2^-122 and have bf16 scales.
template <int FMT, int RT>
__device__ __forceinline__ void tile_by_dots(const Gemv& A, int64_t n0, const uint8_t* lsc, int srow, int lane, int wave,
                                             int nwave) {
  using W = WFmt<FMT>;
  constexpr int PB = W::BLK / 8;                       // code words of a block
  const int words = (int)A.K / 8;
  for (int i = wave; i < 16 * RT * A.M; i += nwave) {
    const int row = i / A.M, m = i % A.M;
    if (n0 + row >= A.N) break;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(A.codes + (n0 + row) * (A.K / 2));
    const u32x4_t* x = reinterpret_cast<const u32x4_t*>(A.x + m * A.ldx);
    float sum = 0.0f;
#pragma unroll 1                                       // no more registers than the usual path
    for (int c = lane; c < words; c += 64) {
      const uint8_t* q = lsc + row * srow + c / PB * (W::SC == 3 ? 2 : 1);
      uint32_t sc;
      if constexpr (W::SC == 3)
        sc = *reinterpret_cast<const uint16_t*>(q);
      else
        sc = *q;
      const u32x4_t xp = x[c];
      const uint32_t w = codes[c];
      float part = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        part = __builtin_amdgcn_fdot2_f32_bf16(decode_pair<false>(w, j), __builtin_bit_cast(bf16x2_t, (uint32_t)xp[j]),
                                               part, false);
      sum = fmaf(part, scale_val(W::SC, sc, 0), sum);
    }
    sum = wave_sum_f(sum);
    if (lane == 0) store_y(A, m, n0 + row, sum);
  }
}

// Orders the LDS accesses of a wave's lanes: LDS serves a wave's instructions
// in order, so only the compiler has to be told.
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// RT tiles of 16 rows per wave, the workgroup's waves splitting K in stages
// of 128 code bytes a row; XT loads bring a stage of the tokens.
template <int FMT, int RT, int XT>
__global__ __launch_bounds__(RT == 1 ? 1024 : 512) void qgemv_mfma_kernel(Gemv A) {
  using W = WFmt<FMT>;
  constexpr int SK = W::FP8 ? 128 : 256;               // K of a stage
  constexpr int XP = SK / 8;                           // 16-byte pieces of a token's stage
  constexpr int HP = XP / 2;                           // and of one half, as it passes through LDS
  constexpr int TPI = 64 / XP;                         // tokens per load
  constexpr int TOK = XT * TPI;
  constexpr int NJ = SK / 32;                          // MFMAs per stage and tile
  constexpr int UB = scale_unit<FMT>();
  extern __shared__ u32x4_t smem[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nwave = blockDim.x >> 6;
  const int r = lane & 15, kg = lane >> 4;
  // all scales of the tile's rows (16 RT srow bytes, one run of memory)
  uint8_t* lsc = reinterpret_cast<uint8_t*>(smem + nwave * (TOK * HP + 128 * RT));
  u32x4_t* lx = smem + wave * (TOK * HP + 128 * RT);        // [TOK][HP] pieces, swizzled by the token
  u32x4_t* lw = lx + TOK * HP;                         // [RT][16][8] pieces, swizzled by the row
  const int K = (int)A.K;
  const int crow = W::FP8 ? K : K / 2, srow = UB * (K / 32);
  const int64_t n0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (16 * RT);
  if (n0 >= A.N) return;                               // the grid's last row is filled up

  __amdgpu_buffer_rsrc_t cb[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t nt = n0 + 16 * t, left = A.N - nt < 16 ? A.N - nt : 16;
    cb[t] = buffer_of(A.codes + nt * crow, left * crow);
  }
  const __amdgpu_buffer_rsrc_t xb = buffer_of(A.x, ((A.M - 1) * A.ldx + K) * 2);

  // lane-linear load positions: codes row lane / 8 (and + 8), tokens lane / XP
  const uint32_t coff = (uint32_t)(lane >> 3) * crow + 16 * (lane & 7);
  const uint32_t xoff = (uint32_t)(lane / XP) * (uint32_t)A.ldx * 2 + 16 * (lane % XP);
  const int nst = (K + SK - 1) / SK;

  u32x4_t wv[RT][2], xv[XT];
  auto load_w = [&](int st) {
    const uint32_t co = 128 * st + 16 * (lane & 7) < crow ? coff + 128 * st : kOutside;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      wv[t][0] = __builtin_amdgcn_raw_buffer_load_b128(cb[t], co, 0, 2);
      wv[t][1] = __builtin_amdgcn_raw_buffer_load_b128(cb[t], co + 8 * crow, 0, 2);
    }
  };
  auto load_x = [&](int st) {
    const int k0 = st * SK;
    const uint32_t xo = k0 + 8 * (lane % XP) < K ? xoff + 2 * k0 : kOutside;
#pragma unroll
    for (int i = 0; i < XT; ++i)
      xv[i] = __builtin_amdgcn_raw_buffer_load_b128(xb, xo + i * TPI * (uint32_t)A.ldx * 2, 0, 0);
  };

  f32x4_t acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  auto swz = [](int tk) { return HP == 16 ? tk : (tk >> 1) & 7; };
  const int tok = r < TOK ? r : TOK - 1;               // columns beyond the tokens are not stored
  load_w(wave);
  load_x(wave);
  if constexpr (UB > 0) {
    const int64_t rows = A.N - n0 < 16 * RT ? A.N - n0 : 16 * RT;
    const int bytes = (int)rows * srow;                // a multiple of 16 in every tile but the last
    const uint8_t* src = A.scales + n0 * srow;         // 16-byte aligned: n0 % 16 == 0
    uint32_t odd = 0u;
    for (int i = threadIdx.x; i < bytes / 16; i += blockDim.x) {
      const u32x4_t v = reinterpret_cast<const u32x4_t*>(src)[i];
      reinterpret_cast<u32x4_t*>(lsc)[i] = v;
      if constexpr (W::SC >= 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) odd |= beyond_bf16<W::SC>(v[j]);
      }
    }
    for (int i = (bytes & ~15) + threadIdx.x; i < 16 * RT * srow; i += blockDim.x) {
      lsc[i] = i < bytes ? src[i] : 0;                 // rows beyond N: zeros
      if constexpr (W::SC == 2)
        if (i < bytes) odd |= beyond_bf16<2>(src[i]);
      if constexpr (W::SC == 3)
        if (i < bytes && i % 2 == 0) odd |= beyond_bf16<3>(src[i] | (uint32_t)src[i + 1] << 8);
    }
    if constexpr (W::SC >= 2) {
      // each wave's word goes into every wave's own pieces, which that wave
      // alone overwrites later: 16 bytes more of LDS would cost a workgroup a
      // CU (E8M0 of 16, 28672 x 8192, 16 tokens: 34.2 us, 41.8 with them)
      const bool any = __any((odd & beyond_mask<W::SC>()) != 0u);
      if (lane < nwave) reinterpret_cast<uint32_t*>(smem + lane * (TOK * HP + 128 * RT))[wave] = any;
      __syncthreads();
      const bool beyond = __any(lane < nwave && reinterpret_cast<const uint32_t*>(lx)[lane < nwave ? lane : 0] != 0u);
      wave_fence();
      if (beyond) {
        tile_by_dots<FMT, RT>(A, n0, lsc, srow, lane, wave, nwave);
        return;
      }
    } else {
      __syncthreads();
    }
  }
  // piece p of a token's stage belongs to k group p / NJ, and to half
  // (p % NJ) / (NJ / 2) of it
  const int xp = lane % XP, hp = xp / NJ * (NJ / 2) + xp % (NJ / 2);
  const bool second = (xp % NJ) / (NJ / 2) != 0;
  auto put_x = [&](bool mine) {
    if (mine) {
#pragma unroll
      for (int i = 0; i < XT; ++i) {
        const int tk = i * TPI + lane / XP;
        lx[tk * HP + (hp ^ swz(tk))] = xv[i];
      }
    }
    wave_fence();
  };
  for (int st = wave; st < nst; st += nwave) {
    const int row = lane >> 3, pc = lane & 7;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      lw[128 * t + row * 8 + (pc ^ (row >> 1))] = wv[t][0];
      lw[128 * t + (row + 8) * 8 + (pc ^ ((row + 8) >> 1 & 7))] = wv[t][1];
    }
    load_w(st + nwave);                                // beyond K: zeros, not used
    const int sk = st * (SK / 32) + kg * (SK / 128);   // the lane's first 32 weights of the stage
    u32x4_t xf[NJ / 2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      put_x(second == (h == 1));
      if (h == 1) load_x(st + nwave);
#pragma unroll
      for (int i = 0; i < NJ / 2; ++i) xf[i] = lx[tok * HP + ((NJ / 2 * kg + i) ^ swz(tok))];
      wave_fence();
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        uint32_t sc = 0u;
        if constexpr (UB > 0) {
          // beyond K the codes are zeros: any scale that is not NaN will do
          const uint8_t* q = lsc + (16 * t + r) * srow + UB * (sk + h < K / 32 ? sk + h : 0);
          if constexpr (UB == 1) sc = *q;
          if constexpr (UB == 2) sc = *reinterpret_cast<const uint16_t*>(q);
          if constexpr (UB == 4) sc = *reinterpret_cast<const uint32_t*>(q);
          if (sk + h >= K / 32) sc = 0u;
        }
        const u32x4_t c = lw[128 * t + r * 8 + ((2 * kg + h) ^ (r >> 1 & 7))];
#pragma unroll
        for (int i = 0; i < NJ / 2; ++i) {
          const float f = UB == 0 ? 1.0f : scale_val(W::SC, sc, i * W::NB / (NJ / 2));
          const bf16x8_t xq = __builtin_bit_cast(bf16x8_t, xf[i]);
          bf16x8_t hi, lo;
          decode8<FMT>(c, i, f, hi, lo);
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, xq, acc[t], 0, 0, 0);
          if constexpr (W::SC == 3) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, xq, acc[t], 0, 0, 0);
        }
      }
    }
    wave_fence();
  }
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);         // [waves][RT * 256]
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[(wave * RT + t) * 256 + q * 64 + lane] = acc[t][q];
  __syncthreads();
  const int e = A.texp ? *A.texp : 0;
  for (int i = threadIdx.x; i < RT * 256; i += blockDim.x) {
    float v = red[i];
    for (int k = 1; k < nwave; ++k) v += red[k * RT * 256 + i];
    const int m = i & 15;
    const int64_t n = n0 + 16 * (i >> 8) + 4 * ((i >> 4) & 3) + ((i >> 6) & 3);
    if (m < A.M && n < A.N) store_y(A, m, n, ldexpf(v, e));
  }
}

namespace {
constexpr size_t kMaxLds = 160 * 1024;
constexpr int64_t kWalkWG = 768;                      // three a CU
constexpr int64_t kPairMost = 1 << 25;                // weights up to which two tokens take the dot form
constexpr int64_t kGridRow = 1 << 20;                 // workgroups of a grid's row: fewer than 2^32 threads

// LDS of a workgroup: the waves' pieces and the tile's scales, or the sums.
template <int FMT>
size_t mfma_lds(int64_t K, int rt, int xt, int waves) {
  const size_t st = (size_t)waves * (xt * 32 + 128 * rt) * 16 + rt * 16 * (size_t)(K / 32) * scale_unit<FMT>();
  const size_t sum = (size_t)waves * rt * 1024;
  return st > sum ? st : sum;
}

template <int FMT, int RT, int XT>
hipError_t gemv_mfma(const Gemv& a, int waves, hipStream_t s) {
  const int64_t wg = ceil_div(a.N, 16 * RT), row = wg < kGridRow ? wg : kGridRow;
  qgemv_mfma_kernel<FMT, RT, XT><<<dim3((unsigned)row, (unsigned)ceil_div(wg, row)), dim3(64 * waves),
                                   mfma_lds<FMT>(a.K, RT, XT, waves), s>>>(a);
  return hipGetLastError();
}

template <int FMT, int MT, bool WALK>
hipError_t gemv_row(const Gemv& a, hipStream_t s) {
  constexpr int64_t step = 64 * WFmt<FMT>::PER, slab = kRowSlab / MT;
  const int64_t held = a.K < slab ? ceil_div(a.K, step) * step : slab;
  int64_t wg = ceil_div(a.N, kRowWaves);
  if (WALK) wg = ceil_div(wg, ceil_div(wg, kWalkWG));  // as many rounds, the same for nearly all
  qgemv_row_kernel<FMT, MT, WALK><<<dim3((unsigned)wg, (unsigned)ceil_div(a.M, MT)), dim3(64 * kRowWaves),
                                    (size_t)held * MT * 2, s>>>(a, wg * kRowWaves);
  return hipGetLastError();
}

template <int FMT>
hipError_t gemv_fmt(const Gemv& a, hipStream_t s) {
  // One token: a row a wave; beyond what is resident the waves stay and walk on,
  // with the token in LDS (28672 x 8192 NVFP4 23.4 us, 28.5 as separate
  // workgroups; 16384 x 4096 8.9 and 11.3; 11008 x 4096 7.2 and 8.3).
  const bool more = a.N > kWalkWG * kRowWaves;
  // Many rows that fill no more than half of a wave's load go to the MFMA form
  // (50000 x 1024: 12.3 us here and 9.8 there; 100000 x 512: 20.5 and 10.3, FP8
  // 17.0 and 13.0), but for bf16 scales, which it pays twice (16384 x 1024: 5.7
  // and 7.1).
  const bool half = WFmt<FMT>::SC != 3 && 2 * a.K <= 64 * WFmt<FMT>::PER;
  if (a.M == 1 && !(more && half))
    return more && a.K <= kRowSlab ? gemv_row<FMT, 1, true>(a, s) : gemv_row<FMT, 1, false>(a, s);
  // Two tokens: the dot form while the time is mostly latency (NVFP4, dot and
  // MFMA: 4096 x 4096 4.7 and 5.3 us, 11264 x 2048 7.0 and 6.1, 28672 x 8192
  // 32.7 and 28.8). With three or four it is never ahead.
  if (a.M == 2 && !more && a.N * a.K <= kPairMost) return gemv_row<FMT, 2, false>(a, s);
  constexpr int TPI = WFmt<FMT>::FP8 ? 4 : 2;          // tokens per load
  const int64_t tiles = ceil_div(a.N, 16), stages = ceil_div(a.K, WFmt<FMT>::FP8 ? 128 : 256);
  // More tiles a wave spare reads of the tokens' values, which are as many
  // bytes as the codes of 64 rows at 16 tokens and next to nothing at 4; but
  // the 256 CUs want a workgroup each, and beyond that two workgroups a CU hide
  // more latency than one with twice the tiles, until the reads weigh more.
  // NVFP4, 16 tokens, one, two, three and four tiles: 4096 x 4096 8.4, 8.9, 10.8,
  // 13.3 us; 7168 x 4096 10.6, 9.5, 11.2, 14.0; 11008 x 4096 14.6, 13.8, 12.1,
  // 14.3; 16384 x 4096 18.7, 14.6, 21.1, 14.8; 28672 x 8192 49.7, 40.3, 48.0, 37.0.
  int rt = a.M <= 4 || tiles <= 256 ? 1 : tiles <= 512 ? 2 : tiles <= 768 ? 3 : tiles <= 1536 ? 2 : 4;
  // Few tiles: more waves along K (2048 x 28672, 3 tokens: 15.3 us with 16
  // waves, 17.1 with 8; 11008 x 4096: 12.2 and 9.4). Four where their loads are
  // long enough: four tiles a wave (28672 x 8192, 16 tokens: 37.4 us with 4,
  // 43.2 with 8), or many workgroups of up to 8 stages a wave (4 tokens, 16384 x
  // 4096: 11.0 us with 4, 11.8 with 8; FP8 28672 x 8192, 16 stages: 41.2 and 39.6).
  const bool few = rt == 4 || (a.M <= 4 && tiles > 768 && stages <= 32);
  int waves = few ? 4 : tiles <= 256 ? 16 : 8;
  if (waves > stages) waves = (int)stages;
  const int xt = a.M <= TPI ? 1 : a.M <= 4 ? 2 : a.M <= 8 ? 8 / TPI : 16 / TPI;
  // The tiles' scales stay in LDS: for a long K fewer tiles, then fewer waves
  // (bf16 scales of 16, 28672 x 28672, 16 tokens: 260 us, 1219 token by token;
  // 24593 x 14400: 152 and 604), and where that does not do, token by token.
  const auto over = [&] { return mfma_lds<FMT>(a.K, rt, xt, waves) > kMaxLds; };
  while (over() && rt > 1) --rt;
  while (over() && waves > 4) waves /= 2;
  if (over()) return gemv_row<FMT, 1, false>(a, s);
  if (a.M <= TPI) return gemv_mfma<FMT, 1, 1>(a, waves, s);
  if constexpr (TPI == 2)
    if (a.M <= 4) return gemv_mfma<FMT, 1, 2>(a, waves, s);
  if (a.M <= 8) {
    if (rt == 1) return gemv_mfma<FMT, 1, 8 / TPI>(a, waves, s);
    if (rt == 2) return gemv_mfma<FMT, 2, 8 / TPI>(a, waves, s);
    if (rt == 3) return gemv_mfma<FMT, 3, 8 / TPI>(a, waves, s);
    return gemv_mfma<FMT, 4, 8 / TPI>(a, waves, s);
  }
  if (rt == 1) return gemv_mfma<FMT, 1, 16 / TPI>(a, waves, s);
  if (rt == 2) return gemv_mfma<FMT, 2, 16 / TPI>(a, waves, s);
  if (rt == 3) return gemv_mfma<FMT, 3, 16 / TPI>(a, waves, s);
  return gemv_mfma<FMT, 4, 16 / TPI>(a, waves, s);
}
}  // namespace

hipError_t launch_gemv(int format, const Gemv& a, hipStream_t s) {
  switch (format) {
    case SNIP_FP8_E4M3: return gemv_fmt<SNIP_FP8_E4M3>(a, s);
    case SNIP_NVFP4: return gemv_fmt<SNIP_NVFP4>(a, s);
    case SNIP_MXFP4: return gemv_fmt<SNIP_MXFP4>(a, s);
    case SNIP_FP4_E4M3_B32: return gemv_fmt<SNIP_FP4_E4M3_B32>(a, s);
    case SNIP_FP4_E8M0_B16: return gemv_fmt<SNIP_FP4_E8M0_B16>(a, s);
    case SNIP_FP4_BF16_B16: return gemv_fmt<SNIP_FP4_BF16_B16>(a, s);
    case SNIP_FP4_BF16_B32: return gemv_fmt<SNIP_FP4_BF16_B32>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace snip
