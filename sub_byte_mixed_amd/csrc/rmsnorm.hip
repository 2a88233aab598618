// RMS norm with the residual's addition, forward (with an optional output
// quantized for the next GEMM) and backward, for gfx950.
//
//   h = x + res, r = 1 / sqrt(mean h^2 + eps), y = h r gamma
//   dx = r (dy gamma - h r mean(dy gamma h r)) + dres, dgamma = sum dy h r
//
// Both are scans bound by HBM: a row is read once, kept in registers over
// its reduction, and written once. TPR threads share a row, each holding VPT
// chunks of 8 elements (chunk t + v TPR, so that a wave's accesses are
// contiguous): with 64 the reduction needs no LDS and a workgroup holds four
// rows, with more it crosses the waves through LDS once per row.
#include "row_common.h"

namespace snip {

// Sum over the threads of a row. `red`: the workgroup's wave sums, one set
// per parity of the call, so that one barrier a call is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[TPR / 64], int parity) {
  v = wave_sum_f(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) red[parity][threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[parity][0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v += red[parity][w];
  }
  return v;
}

// The thread's chunks of a row that starts at element `off`. Chunks beyond
// the row keep what they hold (zeros); a last chunk of cols % 8 elements is
// the business of one thread.
template <int TPR, int VPT, bool F32>
__device__ __forceinline__ void load_row(const void* p, int64_t off, int t, int cols, Raw8<F32> (&r)[VPT]) {
  const int nch = cols >> 3;
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    if (t + v * TPR < nch) load_whole(p, off + 8 * (t + v * TPR), r[v]);
  if ((cols & 7) && t == nch % TPR) {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (v == nch / TPR) load_partial(p, off + 8 * nch, cols & 7, r[v]);
  }
}

// gamma as fp32, from either type: it is read once, after the loads of the
// first row, and waited for here.
template <int TPR, int VPT>
__device__ __forceinline__ void load_gamma(const Mat& m, int t, int cols, float (&g)[VPT][8]) {
  if (m.type == SNIPOP_F32) {
    Raw8<true> r[VPT] = {};
    load_row<TPR>(m.p, 0, t, cols, r);
#pragma unroll
    for (int v = 0; v < VPT; ++v) raw_to_f32(r[v], g[v]);
  } else {
    Raw8<false> r[VPT] = {};
    load_row<TPR>(m.p, 0, t, cols, r);
#pragma unroll
    for (int v = 0; v < VPT; ++v) raw_to_f32(r[v], g[v]);
  }
}

template <int TPR, int VPT>
__device__ __forceinline__ void store_row(const Mat& m, int64_t row, int t, int cols, const float (&x)[VPT][8]) {
  const bool f32 = m.type == SNIPOP_F32;
  const int nch = cols >> 3;
  const int64_t off = row * m.ld;
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    if (t + v * TPR < nch) store_whole(m.p, f32, off + 8 * (t + v * TPR), x[v]);
  if ((cols & 7) && t == nch % TPR) {
    float p[8];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (v == nch / TPR)
        for (int i = 0; i < 8; ++i) p[i] = x[v][i];
    store_partial(m.p, f32, off + 8 * nch, cols & 7, p);
  }
}

constexpr int norm_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

// ------------------------------------------------------------ forward
template <int TPR, int VPT, int PASS, bool XF, bool RF>
__global__ __launch_bounds__(norm_threads(TPR)) void rmsnorm_fwd_kernel(NormFwd A) {
  constexpr int NT = norm_threads(TPR), RPB = NT / TPR, NW = NT / 64;
  constexpr bool QUANT = PASS == SNIP_FP8_E4M3 || PASS == SNIP_NVFP4 || PASS == SNIP_MXFP4;
  __shared__ float red[2][TPR / 64];
  __shared__ uint32_t ured[2 * NW];
  __shared__ double dred[2 * NW];
  __shared__ float inv_lut[PASS == SNIP_NVFP4 ? 128 : 1];
  const int t = threadIdx.x % TPR;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;

  Raw8<XF> rx[VPT] = {};
  Raw8<RF> rr[VPT] = {};
  float g[VPT][8];
  auto load = [&](int64_t i) {
    if (i < A.rows) {
      load_row<TPR>(A.x.p, i * A.x.ld, t, A.cols, rx);
      if (A.res.p) load_row<TPR>(A.res.p, i * A.res.ld, t, A.cols, rr);
    }
  };
  load(row);
  load_gamma<TPR>(A.gamma, t, A.cols, g);

  const int eS = QUANT ? op_tensor_exp<PASS>(A.q, ured) : 0;
  if constexpr (PASS == SNIP_NVFP4) fill_inv_lut(inv_lut);
  const bool stats = QUANT && A.q.part != nullptr;
  const int64_t qch = A.cols >> 3;                 // chunks of a quantized row
  QAcc acc;
  uint32_t amax = 0u;
  for (int it = 0; row < A.rows; ++it, row += step) {
    float h[VPT][8];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float b[8];
      raw_to_f32(rx[v], h[v]);
      raw_to_f32(rr[v], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (A.res.p) h[v][i] += b[i];
        ss = fmaf(h[v][i], h[v][i], ss);
      }
    }
    load(row + step);
    ss = row_sum<TPR>(ss, red, it & 1);
    const float r = 1.0f / sqrtf(ss / (float)A.cols + A.eps);
    if constexpr (PASS != kPassAmax) {
      if (A.h.p) store_row<TPR>(A.h, row, t, A.cols, h);
      if (A.rstd && t == 0) A.rstd[row] = r;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * r * g[v][i];
    if constexpr (PASS == kPassAmax) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (8 * (t + v * TPR) < A.cols) amax = chunk_max_bits(h[v], amax);
    } else {
      if (A.y.p) store_row<TPR>(A.y, row, t, A.cols, h);
      if constexpr (QUANT) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
          if (t + v * TPR < qch) quant_chunk<PASS>(A.q, eS, inv_lut, row * qch + t + v * TPR, h[v], stats, acc);
      }
    }
  }
  if constexpr (PASS == kPassAmax) {
    amax = wg_max_u(amax, ured);
    if (threadIdx.x == 0) A.amax_out[blockIdx.x] = amax;
  }
  if constexpr (QUANT) {
    if (stats)
      wg_store_stats(A.q.part + blockIdx.x, ldexp(acc.e2s, 2 * eS) + acc.e2r, ldexp(acc.x2s, 2 * eS) + acc.x2r,
                     acc.nf, acc.tmax, dred, ured);
  }
}

// ------------------------------------------------------------ backward
// A thread's columns stay the same over the workgroup's rows, so dgamma is
// summed in registers; each workgroup leaves one partial row, and a second
// launch sums those in a fixed order (no atomics: the result does not depend
// on timing).
template <int TPR, int VPT, bool YF, bool HF, bool RF>
__global__ __launch_bounds__(norm_threads(TPR)) void rmsnorm_bwd_kernel(NormBwd A) {
  constexpr int NT = norm_threads(TPR), RPB = NT / TPR;
  __shared__ float red[2][TPR / 64];
  __shared__ float lds[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? VPT * 8 * TPR : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + sub;

  Raw8<YF> ry[VPT] = {};
  Raw8<HF> rh[VPT] = {};
  Raw8<RF> rr[VPT] = {};
  float g[VPT][8];
  float rs = 0.0f;
  auto load = [&](int64_t i) {
    if (i < A.rows) {
      load_row<TPR>(A.dy.p, i * A.dy.ld, t, A.cols, ry);
      load_row<TPR>(A.h.p, i * A.h.ld, t, A.cols, rh);
      if (A.dres.p) load_row<TPR>(A.dres.p, i * A.dres.ld, t, A.cols, rr);
      rs = A.rstd[i];
    }
  };
  load(row);
  load_gamma<TPR>(A.gamma, t, A.cols, g);
  float dg[VPT][8];
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[v][i] = 0.0f;

  for (int it = 0; row < A.rows; ++it, row += step) {
    float d[VPT][8], xh[VPT][8], res[VPT][8];
    const float r = rs;
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      raw_to_f32(ry[v], d[v]);
      raw_to_f32(rh[v], xh[v]);
      raw_to_f32(rr[v], res[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[v][i] *= r;
        dg[v][i] = fmaf(d[v][i], xh[v][i], dg[v][i]);
        d[v][i] *= g[v][i];
        dot = fmaf(d[v][i], xh[v][i], dot);
      }
    }
    load(row + step);
    const float mean = row_sum<TPR>(dot, red, it & 1) / (float)A.cols;
    if (A.dx.p) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[v][i] = r * fmaf(-xh[v][i], mean, d[v][i]);
          if (A.dres.p) d[v][i] += res[v][i];
        }
      store_row<TPR>(A.dx, row, t, A.cols, d);
    }
  }
  if (!A.part) return;
  if constexpr (RPB > 1) {
    if (sub > 0) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) lds[sub - 1][(v * 8 + i) * TPR + t] = dg[v][i];
    }
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int s = 0; s < RPB - 1; ++s)
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[v][i] += lds[s][(v * 8 + i) * TPR + t];
  }
  float* dst = A.part + (int64_t)blockIdx.x * A.part_ld;
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    if (8 * (t + v * TPR) < A.part_ld) store_whole(dst, true, 8 * (t + v * TPR), dg[v]);
}

// dgamma[c] = sum over the workgroups' partial rows: 16 threads x 4 columns,
// 16 slices of the rows joined through LDS.
__global__ __launch_bounds__(256) void dgamma_sum_kernel(const float* part, int64_t ld, int nwg, int cols,
                                                         float* dgamma) {
  __shared__ float4 red[16][16];
  const int cx = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int64_t c = ((int64_t)blockIdx.x * 16 + cx) * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < ld) {
#pragma unroll 4
    for (int i = slice; i < nwg; i += 16) {
      const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)i * ld + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  red[slice][cx] = s;
  __syncthreads();
  if (slice == 0 && c < ld) {
    for (int k = 1; k < 16; ++k) {
      const float4 v = red[k][cx];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    const float o[4] = {s.x, s.y, s.z, s.w};
    for (int i = 0; i < 4; ++i)
      if (c + i < cols) dgamma[c + i] = o[i];
  }
}

// ------------------------------------------------------------ shapes
namespace {
struct NormShape {
  int tpr, vpt;
};

// One chunk a thread up to 2048 columns, two beyond: with four, the fp32
// forms need 170 to 256 VGPRs and scratch.
NormShape norm_shape(int64_t cols) {
  const int64_t ch = ceil_div(cols, 8);
  if (ch <= 64) return {64, 1};
  if (ch <= 256) return {256, 1};
  if (ch <= 512) return {256, 2};
  if (ch <= 1024) return {512, 2};
  return {1024, 2};
}

int norm_wg(int64_t rows, int64_t cols, int most) {
  const NormShape s = norm_shape(cols);
  const int64_t wg = ceil_div(rows, norm_threads(s.tpr) / s.tpr);
  return (int)(wg < most ? wg : most);
}

// f(shape constants) for the row's shape.
template <class F>
void with_shape(int64_t cols, F f) {
  const NormShape k = norm_shape(cols);
  using std::integral_constant;
  if (k.tpr == 64) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (k.vpt == 1) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (k.tpr == 256) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  if (k.tpr == 512) return f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
}

// f(F32) for a matrix's type; an absent one counts as bf16.
template <class F>
void with_type(const Mat& m, F f) {
  if (m.p && m.type == SNIPOP_F32) return f(std::true_type{});
  return f(std::false_type{});
}

template <int PASS>
hipError_t norm_fwd_pass(const NormFwd& a, int nwg, hipStream_t s) {
  with_shape(a.cols, [&](auto tpr, auto vpt) {
    with_type(a.x, [&](auto xf) {
      with_type(a.res, [&](auto rf) {
        constexpr int T = decltype(tpr)::value, V = decltype(vpt)::value;
        rmsnorm_fwd_kernel<T, V, PASS, decltype(xf)::value, decltype(rf)::value>
            <<<dim3(nwg), dim3(norm_threads(T)), 0, s>>>(a);
      });
    });
  });
  return hipGetLastError();
}
}  // namespace

int norm_fwd_wg(int64_t rows, int64_t cols, bool amax) { return norm_wg(rows, cols, amax ? kOpsAmaxWG : kOpsWG); }
int norm_bwd_wg(int64_t rows, int64_t cols) { return norm_wg(rows, cols, 512); }

hipError_t launch_norm_fwd(int pass, const NormFwd& a, int nwg, hipStream_t s) {
  switch (pass) {
    case kPassAmax: return norm_fwd_pass<kPassAmax>(a, nwg, s);
    case SNIP_FP8_E4M3: return norm_fwd_pass<SNIP_FP8_E4M3>(a, nwg, s);
    case SNIP_NVFP4: return norm_fwd_pass<SNIP_NVFP4>(a, nwg, s);
    case SNIP_MXFP4: return norm_fwd_pass<SNIP_MXFP4>(a, nwg, s);
    default: return norm_fwd_pass<SNIP_BF16>(a, nwg, s);
  }
}

hipError_t launch_norm_bwd(const NormBwd& a, float* dgamma, int nwg, hipStream_t s) {
  with_shape(a.cols, [&](auto tpr, auto vpt) {
    with_type(a.dy, [&](auto yf) {
      with_type(a.h, [&](auto hf) {
        with_type(a.dres, [&](auto rf) {
          constexpr int T = decltype(tpr)::value, V = decltype(vpt)::value;
          rmsnorm_bwd_kernel<T, V, decltype(yf)::value, decltype(hf)::value, decltype(rf)::value>
              <<<dim3(nwg), dim3(norm_threads(T)), 0, s>>>(a);
        });
      });
    });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dgamma) return e;
  dgamma_sum_kernel<<<dim3((unsigned)ceil_div(a.part_ld, 64)), dim3(256), 0, s>>>(a.part, a.part_ld, nwg, a.cols,
                                                                                 dgamma);
  return hipGetLastError();
}

}  // namespace snip
