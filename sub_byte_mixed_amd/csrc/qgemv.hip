// y[M][N] = x[M][K] . dequant(w)[N][K]^T for 1..16 tokens, gfx950.
//
//   y[m][n] = 2^e sum_b s[n][b] sum_{k in block b} c[n][k] x[m][k]
//
// Bound by the weights' bytes (0.53 to 1 byte each). A lane loads 16 bytes of
// codes of a row (32 E2M1 or 16 E4M3 weights), decodes them to bf16 pairs
// (exact: 2 or 4 significant bits) and multiplies them with the tokens' bf16
// by v_dot2_f32_bf16: exact products, fp32 sums. The block scale multiplies
// the block's sum, so it costs one operation a block.
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

// The scales of the NB blocks of chunk `c` (PER weights) of row `n`.
template <int FMT>
__device__ __forceinline__ uint32_t load_scales(const Gemv& A, int64_t n, int64_t c) {
  using W = WFmt<FMT>;
  if constexpr (W::SC == 0) return 0u;
  const int64_t i = (n * (A.K / W::PER) + c) * W::NB;  // K % PER == 0
  if constexpr (W::SC == 3) {
    if constexpr (W::NB == 2) return *reinterpret_cast<const uint32_t*>(A.scales + 2 * i);
    return *reinterpret_cast<const uint16_t*>(A.scales + 2 * i);
  }
  if constexpr (W::NB == 2) return *reinterpret_cast<const uint16_t*>(A.scales + i);
  return A.scales[i];
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

// One wave per row, one token per blockIdx.y. Bound by the vector memory
// unit rather than by HBM (a lane's 64 bytes of x are four scattered
// accesses), but with nothing to set up: 2.2 us for 256 x 2048 where the MFMA
// form takes 3.4, 3.0 for 2048 x 2048 (3.8); behind from 2^23 weights on
// (4096 x 11008: 10 us for 8.5).
template <int FMT>
__global__ __launch_bounds__(256) void qgemv_dot_kernel(Gemv A) {
  using W = WFmt<FMT>;
  const int lane = threadIdx.x & 63;
  const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int m = blockIdx.y;
  if (n >= A.N) return;
  const int64_t nch = A.K / W::PER;
  const uint8_t* codes = A.codes + n * (W::FP8 ? A.K : A.K / 2);
  const uint16_t* xm = A.x + m * A.ldx;
  float acc = 0.0f;
  for (int64_t c = lane; c < nch; c += 64) {
    const u32x4_t w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(codes + 16 * c));
    const uint32_t sc = load_scales<FMT>(A, n, c);
    const u32x4_t* xp = reinterpret_cast<const u32x4_t*>(xm + c * W::PER);
    float part[W::NB];
#pragma unroll
    for (int b = 0; b < W::NB; ++b) part[b] = 0.0f;
#pragma unroll
    for (int q = 0; q < W::PER / 8; ++q) {
      const u32x4_t x = xp[q];                         // values of the pairs 4q .. 4q+3
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int pair = 4 * q + j, per = W::FP8 ? 2 : 4;
        float& p = part[pair * 2 * W::NB / W::PER];
        p = __builtin_amdgcn_fdot2_f32_bf16(decode_pair<W::FP8>(w[pair / per], pair % per),
                                            __builtin_bit_cast(bf16x2_t, (uint32_t)x[j]), p, false);
      }
    }
#pragma unroll
    for (int b = 0; b < W::NB; ++b)
      acc = W::SC == 0 ? acc + part[b] : fmaf(part[b], scale_val(W::SC, sc, b), acc);
  }
  const float v = wave_sum_f(acc);
  if (lane == 0) store_y(A, m, n, ldexpf(v, A.texp ? *A.texp : 0));
}

// ------------------------------------------------------------ MFMA form
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// 8 weights (one code word of E2M1, two of E4M3) with their block scale ->
// 8 bf16. E4M3 codes, and E2M1 times an E4M3 or E8M0 scale (6 and 2
// significant bits), are exact in bf16. E2M1 times a bf16 scale has up to 9
// bits: it is the exact sum of `hi` and `lo`.
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

// Buffer descriptor over `bytes` of p: a load whose offset lies beyond them
// returns zero, which stands in for rows and columns outside the operands.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(bytes > 0 ? bytes : 0), 0x00027000);
}
// Orders the LDS accesses of a wave's lanes: LDS serves a wave's instructions
// in order, so only the compiler has to be told.
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }
constexpr uint32_t kOutside = 0x80000000u;             // beyond every descriptor

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
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);

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
  auto load = [&](int st) {
    const int k0 = st * SK;
    const uint32_t co = 128 * st + 16 * (lane & 7) < crow ? coff + 128 * st : kOutside;
    const uint32_t xo = k0 + 8 * (lane % XP) < K ? xoff + 2 * k0 : kOutside;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      wv[t][0] = __builtin_amdgcn_raw_buffer_load_b128(cb[t], co, 0, 2);
      wv[t][1] = __builtin_amdgcn_raw_buffer_load_b128(cb[t], co + 8 * crow, 0, 2);
    }
#pragma unroll
    for (int i = 0; i < XT; ++i)
      xv[i] = __builtin_amdgcn_raw_buffer_load_b128(xb, xo + i * TPI * (uint32_t)A.ldx * 2, 0, 0);
  };

  f32x4_t acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  auto swz = [](int tk) { return HP == 16 ? tk : (tk >> 1) & 7; };
  const int tok = r < TOK ? r : TOK - 1;               // columns beyond the tokens are not stored
  load(wave);
  if constexpr (UB > 0) {
    const int64_t rows = A.N - n0 < 16 * RT ? A.N - n0 : 16 * RT;
    const int bytes = (int)rows * srow;                // a multiple of 16 in every tile but the last
    const uint8_t* src = A.scales + n0 * srow;         // 16-byte aligned: n0 % 16 == 0
    for (int i = threadIdx.x; i < bytes / 16; i += blockDim.x)
      reinterpret_cast<u32x4_t*>(lsc)[i] = reinterpret_cast<const u32x4_t*>(src)[i];
    for (int i = (bytes & ~15) + threadIdx.x; i < 16 * RT * srow; i += blockDim.x)
      lsc[i] = i < bytes ? src[i] : 0;                 // rows beyond N: zeros
    __syncthreads();
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
    const int sk = st * (SK / 32) + kg * (SK / 128);   // the lane's first 32 weights of the stage
    u32x4_t xf[NJ / 2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      put_x(second == (h == 1));
      if (h == 1) load(st + nwave);                    // beyond K: zeros, not used
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

// LDS of a workgroup: the waves' pieces and the tile's scales, or the sums.
template <int FMT>
size_t mfma_lds(int64_t K, int rt, int xt, int waves) {
  const size_t st = (size_t)waves * (xt * 32 + 128 * rt) * 16 + rt * 16 * (size_t)(K / 32) * scale_unit<FMT>();
  const size_t sum = (size_t)waves * rt * 1024;
  return st > sum ? st : sum;
}

template <int FMT, int RT, int XT>
hipError_t gemv_mfma(const Gemv& a, int waves, hipStream_t s) {
  qgemv_mfma_kernel<FMT, RT, XT><<<dim3((unsigned)ceil_div(a.N, 16 * RT)), dim3(64 * waves),
                                   mfma_lds<FMT>(a.K, RT, XT, waves), s>>>(a);
  return hipGetLastError();
}

template <int FMT>
hipError_t gemv_fmt(const Gemv& a, hipStream_t s) {
  constexpr int TPI = WFmt<FMT>::FP8 ? 4 : 2;          // tokens per load
  const int64_t tiles = ceil_div(a.N, 16), stages = ceil_div(a.K, WFmt<FMT>::FP8 ? 128 : 256);
  // More rows a wave spare reads of the tokens' values, which are as many
  // bytes as the codes of 64 rows at 16 tokens and next to nothing at 4; but
  // the 256 CUs want a workgroup each. Few tiles: more waves along K.
  const int rt = a.M <= 4 || tiles < 512 ? 1 : tiles < 1024 ? 2 : 4;
  int waves = rt == 4 ? 4 : tiles <= 256 ? 16 : 8;
  if (waves > stages) waves = (int)stages;
  const int xt = a.M <= TPI ? 1 : a.M <= 4 ? 2 : a.M <= 8 ? 8 / TPI : 16 / TPI;
  if ((a.M == 1 && a.N * a.K <= (int64_t)1 << 23) || mfma_lds<FMT>(a.K, rt, xt, waves) > kMaxLds) {
    qgemv_dot_kernel<FMT><<<dim3((unsigned)ceil_div(a.N, 4), a.M), dim3(256), 0, s>>>(a);
    return hipGetLastError();
  }
  if (a.M <= TPI) return gemv_mfma<FMT, 1, 1>(a, waves, s);
  if constexpr (TPI == 2)
    if (a.M <= 4) return gemv_mfma<FMT, 1, 2>(a, waves, s);
  if (a.M <= 8) {
    if (rt == 1) return gemv_mfma<FMT, 1, 8 / TPI>(a, waves, s);
    if (rt == 2) return gemv_mfma<FMT, 2, 8 / TPI>(a, waves, s);
    return gemv_mfma<FMT, 4, 8 / TPI>(a, waves, s);
  }
  if (rt == 1) return gemv_mfma<FMT, 1, 16 / TPI>(a, waves, s);
  if (rt == 2) return gemv_mfma<FMT, 2, 16 / TPI>(a, waves, s);
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
