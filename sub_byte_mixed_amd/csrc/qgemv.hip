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

__device__ __forceinline__ float scale_val(int sc, uint32_t raw, int i) {
  if (sc == 3) return __uint_as_float((raw >> (16 * i)) << 16);
  const uint32_t b = (raw >> (8 * i)) & 0xFFu;
  if (sc == 1) return __builtin_amdgcn_cvt_f32_fp8((int)b, 0);
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

// One wave per row n, the workgroup's four waves on four rows; tokens in
// groups of MT (blockIdx.y).
template <int FMT, int MT>
__global__ __launch_bounds__(256) void qgemv_dot_kernel(Gemv A) {
  using W = WFmt<FMT>;
  const int lane = threadIdx.x & 63;
  const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int m0 = blockIdx.y * MT;
  if (n >= A.N) return;
  const int64_t nch = A.K / W::PER;
  const uint8_t* codes = A.codes + n * (W::FP8 ? A.K : A.K / 2);
  float acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = 0.0f;
  for (int64_t c = lane; c < nch; c += 64) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(codes + 16 * c);
    const uint32_t sc = load_scales<FMT>(A, n, c);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int mm = m0 + m < A.M ? m0 + m : A.M - 1;
      const u32x4_t* xp = reinterpret_cast<const u32x4_t*>(A.x + mm * A.ldx + c * W::PER);
      float part[W::NB];
#pragma unroll
      for (int b = 0; b < W::NB; ++b) part[b] = 0.0f;
#pragma unroll
      for (int q = 0; q < W::PER / 8; ++q) {
        const u32x4_t x = xp[q];                       // 8 tokens' values: pairs 4q .. 4q+3
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
        acc[m] = W::SC == 0 ? acc[m] + part[b] : fmaf(part[b], scale_val(W::SC, sc, b), acc[m]);
    }
  }
  const int e = A.texp ? *A.texp : 0;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float v = acc[m];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    if (lane == 0 && m0 + m < A.M) store_y(A, m0 + m, n, ldexpf(v, e));
  }
}

namespace {
template <int FMT>
hipError_t gemv_fmt(const Gemv& a, hipStream_t s) {
  const unsigned gx = (unsigned)ceil_div(a.N, 4);
  if (a.M == 1)
    qgemv_dot_kernel<FMT, 1><<<dim3(gx, 1), dim3(256), 0, s>>>(a);
  else
    qgemv_dot_kernel<FMT, 4><<<dim3(gx, (unsigned)ceil_div(a.M, 4)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
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
