// Device helpers of the row operators (rmsnorm.hip, swiglu.hip): a thread
// works on chunks of E consecutive elements, so that an access is 16 bytes
// where it can be and an E2M1 block lies in the chunks of a few neighbouring
// lanes.
#pragma once

#include <type_traits>

#include "ops.h"
#include "quant_common.h"

namespace snip {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// A chunk of E elements as loaded. The conversion is left to the use, so that
// the loads of several chunks are in flight at once. The type is a template
// argument: with a type tested at run time the compiler keeps both forms
// alive (126 VGPRs where 50 do).
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
template <bool F32, int E = 8>
struct Raw {
  static constexpr int BYTES = E * (F32 ? 4 : 2), NV = BYTES / 16;
  u32x4_t w[NV ? NV : 1];      // 8 bytes: the first two words
};

template <bool F32, int E>
__device__ __forceinline__ void raw_to_f32(const Raw<F32, E>& r, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if constexpr (F32)
      x[i] = __uint_as_float(r.w[i / 4][i % 4]);
    else
      x[i] = i % 2 ? bf16_hi(r.w[0][i / 2]) : bf16_lo(r.w[0][i / 2]);
  }
}

// Whole chunk at element offset `off` of `p`; NT: read past the caches.
template <bool NT = false, bool F32, int E>
__device__ __forceinline__ void load_whole(const void* p, int64_t off, Raw<F32, E>& r) {
  const uint8_t* b = static_cast<const uint8_t*>(p) + off * (F32 ? 4 : 2);
  if constexpr (Raw<F32, E>::NV == 0) {
    const u32x2_t* q = reinterpret_cast<const u32x2_t*>(b);
    const u32x2_t v = NT ? __builtin_nontemporal_load(q) : *q;
    r.w[0][0] = v[0];
    r.w[0][1] = v[1];
  } else {
    const u32x4_t* q = reinterpret_cast<const u32x4_t*>(b);
#pragma unroll
    for (int k = 0; k < Raw<F32, E>::NV; ++k) r.w[k] = NT ? __builtin_nontemporal_load(q + k) : q[k];
  }
}

// The first n < E elements of a chunk, the others zero: element loads, since
// a row's last chunk may end where the allocation does.
template <bool F32, int E>
__device__ __forceinline__ void load_partial(const void* p, int64_t off, int n, Raw<F32, E>& r) {
  r = {};
#pragma unroll
  for (int i = 0; i < E - 1; ++i) {
    if (i < n) {
      if constexpr (F32)
        r.w[i / 4][i % 4] = static_cast<const uint32_t*>(p)[off + i];
      else
        r.w[0][i / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[off + i] << (16 * (i % 2));
    }
  }
}

// Two fp32 -> packed bf16, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2_t v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

template <int E>
__device__ __forceinline__ void store_whole(void* p, bool f32, int64_t off, const float (&x)[E]) {
  if (f32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + off);
#pragma unroll
    for (int k = 0; k < E / 4; ++k) q[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
  } else if constexpr (E == 8) {
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + off) =
        u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
  } else {
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(p) + off) = u32x2_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
  }
}

template <int E>
__device__ inline void store_partial(void* p, bool f32, int64_t off, int n, const float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E - 1; ++i) {
    if (i < n) {
      if (f32)
        static_cast<float*>(p)[off + i] = x[i];
      else
        static_cast<uint16_t*>(p)[off + i] = (uint16_t)pack_bf16(x[i], 0.0f);
    }
  }
}

// Maximum over the groups of LANES (2, 4 or 8) neighbouring lanes, in each of
// them: DPP moves, no LDS.
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
  auto step = [](float x, auto ctrl) {
    return fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xF, 0xF,
                                                               true)));
  };
  v = step(v, std::integral_constant<int, 0xB1>{});                             // lane ^ 1
  if constexpr (LANES > 2) v = step(v, std::integral_constant<int, 0x4E>{});    // lane ^ 2
  if constexpr (LANES > 4) v = step(v, std::integral_constant<int, 0x141>{});   // mirror of 8
  return v;
}

// Sum over the wave, in every lane: four steps within rows of 16 lanes, then
// the four row sums.
__device__ __forceinline__ float wave_sum_f(float v) {
  auto step = [](float x, auto ctrl) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v = step(v, std::integral_constant<int, 0xB1>{});    // lane ^ 1
  v = step(v, std::integral_constant<int, 0x4E>{});    // lane ^ 2
  v = step(v, std::integral_constant<int, 0x141>{});   // mirror of 8
  v = step(v, std::integral_constant<int, 0x140>{});   // mirror of 16
  const int b = __float_as_int(v);
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(b, 0));
  const float r1 = __int_as_float(__builtin_amdgcn_readlane(b, 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(b, 32));
  const float r3 = __int_as_float(__builtin_amdgcn_readlane(b, 48));
  return (r0 + r1) + (r2 + r3);
}

// Statistics of one thread's quantized chunks.
struct QAcc {
  double e2s = 0.0, x2s = 0.0;      // tensor-scaled domain (NVFP4, FP8)
  double e2r = 0.0, x2r = 0.0;      // raw domain (MX, chunks of non-finite blocks)
  uint32_t nf = 0u, tmax = 0u;
};

// Quantize one chunk y of E values, chunk index `g` of the output layout
// (row * K / E + chunk of the row), with the rules of snip_quantize on the
// fp32 values. The lanes that share a block hold its chunks in order, are
// active together, and start at a multiple of their number. Statistics only
// where `stats` (uniform) asks for them.
template <int FMT, bool SR, int E>
__device__ __forceinline__ void quant_chunk(const OpQuant& Q, int eS, const float* inv_lut, int64_t g,
                                            const float (&y)[E], bool stats, QAcc& acc) {
  constexpr int LANES = (FMT == SNIP_MXFP4 ? 32 : 16) / E;      // of a block
  constexpr int W = E / 4;
  float r[8];                       // the upper half unused where E is 4
  float shat = 1.0f;                // NVFP4: decoded block scale
  int X = 0;                        // MX: scale exponent
  Words4 d;
  if constexpr (SR) {
    d = draws8(Q.seed, Q.tensor_id, (uint64_t)(E == 8 ? g : g >> 1));
    if (E == 4 && (g & 1)) {        // the block's second half: its words to the front
      d.w[0] = d.w[2];
      d.w[1] = d.w[3];
    }
  }
  float xs[E];                      // the scaled values that the error refers to
  uint32_t code[W];
  if constexpr (FMT == SNIP_FP8_E4M3) {
    float c[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      xs[i] = ldexpf(y[i], -eS);
      c[i] = __builtin_amdgcn_fmed3f(xs[i], -448.0f, 448.0f);
    }
#pragma unroll
    for (int k = 0; k < W; ++k) code[k] = SR ? fp8x4_sr(c + 4 * k, d, 4 * k) : fp8x4_rne(c + 4 * k);
    if constexpr (E == 8)
      *reinterpret_cast<u32x2_t*>(Q.codes + g * 8) = u32x2_t{code[0], code[W - 1]};
    else
      *reinterpret_cast<uint32_t*>(Q.codes + g * 4) = code[0];
  } else {
    float am = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      xs[i] = FMT == SNIP_NVFP4 ? ldexpf(y[i], -eS) : y[i];
      am = fmaxf(am, fabsf(xs[i]));
    }
    am = group_max<LANES>(am);
    uint32_t sc;
    if constexpr (FMT == SNIP_NVFP4) {
      sc = e4m3_rne(am / 6.0f);
      shat = e4m3_val(sc);
      const float inv = inv_lut[sc];
#pragma unroll
      for (int i = 0; i < E; ++i) r[i] = xs[i] * inv;
    } else {
      X = -127;
      if (am > 0.0f) {
        X = (int)(__float_as_uint(am) >> 23) - 129;      // floor(log2 am) - 2
        X = X < -127 ? -127 : X;
      }
      sc = (uint32_t)(X + 127);
      const float pw = am > 0.0f ? exp2i(-X) : 0.0f;
#pragma unroll
      for (int i = 0; i < E; ++i) xs[i] = r[i] = y[i] * pw;
    }
    if (threadIdx.x % LANES == 0) Q.scales[g / LANES] = (uint8_t)sc;
    if constexpr (E == 4) r[4] = r[5] = r[6] = r[7] = 0.0f;
    code[0] = SR ? fp4x8_sr(r, d) : fp4x8_rne(r);
    if constexpr (E == 8)
      *reinterpret_cast<uint32_t*>(Q.codes + g * 4) = code[0];
    else
      *reinterpret_cast<uint16_t*>(Q.codes + g * 2) = (uint16_t)code[0];
  }
  if (!stats) return;
  float q[8];
  if constexpr (FMT == SNIP_FP8_E4M3) {
#pragma unroll
    for (int k = 0; k < W; ++k) fp8x4_dec(code[k], q + 4 * k);
  } else {
    fp4x8_dec(code[0], q);
  }
  float be2 = 0.0f, bx2 = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float err = FMT == SNIP_NVFP4 ? fmaf(q[i], shat, -xs[i]) : q[i] - xs[i];
    be2 = fmaf(err, err, be2);
    bx2 = fmaf(xs[i], xs[i], bx2);
  }
  // a block with a non-finite value has no error to report: its lanes agree
  float bad = bx2 <= 3.0e38f ? 0.0f : 1.0f;
  if constexpr (FMT != SNIP_FP8_E4M3) bad = group_max<LANES>(bad);
  if (bad != 0.0f) {
    uint32_t nf = 0u, am = 0u;
    double x2 = 0.0;
    nonfinite_stats<E>(y, nf, x2, am);
    acc.nf += nf;
    acc.x2r += x2;
    acc.tmax = max(acc.tmax, am);
    return;
  }
  acc.tmax = max(acc.tmax, block_absmax_bits<E>(y));
  if constexpr (FMT == SNIP_MXFP4) {
    acc.e2r += ldexp((double)be2, 2 * X);
    acc.x2r += ldexp((double)bx2, 2 * X);
  } else {
    acc.e2s += (double)be2;
    acc.x2s += (double)bx2;
  }
}

// Finite max |y| of a chunk as fp32 bits.
template <int E>
__device__ __forceinline__ uint32_t chunk_max_bits(const float (&y)[E], uint32_t m) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint32_t b = __float_as_uint(y[i]) & 0x7FFFFFFFu;
    const uint32_t v = b < 0x7F800000u ? b : 0u;
    m = v > m ? v : m;
  }
  return m;
}

// Maximum over the workgroup (all threads get it); red: one word per wave.
__device__ inline uint32_t wg_max_u(uint32_t m, uint32_t* red) {
  m = wave_max_u(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = red[0];
  for (int w = 1; w < (int)(blockDim.x >> 6); ++w) m = red[w] > m ? red[w] : m;
  __syncthreads();
  return m;
}

// Tensor exponent of a quantized output: from the supplied max, or from the
// partials of the pass for the maximum.
template <int FMT>
__device__ inline int op_tensor_exp(const OpQuant& Q, uint32_t* red) {
  if constexpr (FMT == SNIP_FP8_E4M3 || FMT == SNIP_NVFP4) {
    float A;
    if (Q.amax_in) {
      A = *Q.amax_in;
    } else {
      uint32_t m = 0u;
      for (int i = threadIdx.x; i < Q.n_amax_part; i += blockDim.x) m = max(m, Q.amax_part[i]);
      A = __uint_as_float(wg_max_u(m, red));
    }
    const int e = tensor_exp(A, FMT);
    if (blockIdx.x == 0 && threadIdx.x == 0) *Q.texp = e;
    return e;
  }
  return 0;
}

}  // namespace snip
