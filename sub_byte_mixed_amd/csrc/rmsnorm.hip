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
// Measured, calls back to back: forward 4096 x 2048, fp32 x, bf16 residual, to
// bf16 and FP8 with statistics, 22.2 us (4.2 TB/s); 4096 x 8192, bf16, to FP8,
// 43.8 us (5.4 TB/s, a large copy's rate); backward 4096 x 2048, fp32 dy, 18.4 us
// (4.6 TB/s, with dgamma's second launch). Finding the maximum itself is one more
// pass over the inputs: 4096 x 2048 24.0 -> 35.5 us in a graph, 4096 x 8192 48.6 ->
// 75.6; NVFP4 and MX-FP4 outputs take 1 to 2 us less than FP8.
#include "row_common.h"

namespace snip {

// Sum over the threads of a row, which are the workgroup's (WG) or a wave's.
// `red`: the workgroup's wave sums, one set per parity of the call, so that
// one barrier a call is enough.
template <bool WG>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int parity) {
  v = wave_sum_f(v);
  if constexpr (WG) {
    if ((threadIdx.x & 63) == 0) red[parity][threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[parity][0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) v += red[parity][w];
  }
  return v;
}

// The thread's chunks of a row that starts at element `off`. Chunks beyond
// the row keep what they hold (zeros); a last chunk of cols % 8 elements is
// the business of one thread.
template <int VPT, bool F32>
__device__ __forceinline__ void load_row(const void* p, int64_t off, int t, int tpr, int cols, Raw<F32> (&r)[VPT]) {
  const int nch = cols >> 3;
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    if (t + v * tpr < nch) load_whole(p, off + 8 * (t + v * tpr), r[v]);
  if ((cols & 7) && t == nch % tpr) {
    Raw<F32> last;
    load_partial(p, off + 8 * nch, cols & 7, last);
#pragma unroll
    for (int k = 0; k < Raw<F32>::NV; ++k) {
      // a value from here on: the compiler would choose among the chunks'
      // addresses, and keep them in scratch for it (twice the time)
      asm("" : "+v"(last.w[k]));
#pragma unroll
      for (int v = 0; v < VPT; ++v) r[v].w[k] = v == nch / tpr ? last.w[k] : r[v].w[k];
    }
  }
}

// gamma as fp32, from either type: it is read once, after the loads of the
// first row, and waited for here.
template <int VPT>
__device__ __forceinline__ void load_gamma(const Mat& m, int t, int tpr, int cols, float (&g)[VPT][8]) {
  if (m.type == SNIPOP_F32) {
    Raw<true> r[VPT] = {};
    load_row(m.p, 0, t, tpr, cols, r);
#pragma unroll
    for (int v = 0; v < VPT; ++v) raw_to_f32(r[v], g[v]);
  } else {
    Raw<false> r[VPT] = {};
    load_row(m.p, 0, t, tpr, cols, r);
#pragma unroll
    for (int v = 0; v < VPT; ++v) raw_to_f32(r[v], g[v]);
  }
}

template <int VPT>
__device__ __forceinline__ void store_row(const Mat& m, int64_t row, int t, int tpr, int cols, const float (&x)[VPT][8]) {
  const bool f32 = m.type == SNIPOP_F32;
  const int nch = cols >> 3;
  const int64_t off = row * m.ld;
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    if (t + v * tpr < nch) store_whole(m.p, f32, off + 8 * (t + v * tpr), x[v]);
  if ((cols & 7) && t == nch % tpr) {
    float p[8];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (v == nch / tpr)
        for (int i = 0; i < 8; ++i) p[i] = x[v][i];
    store_partial(m.p, f32, off + 8 * nch, cols & 7, p);
  }
}

// A row to a workgroup (WG), or to each of a workgroup's four waves.
template <bool WG>
struct RowMap {
  int t, tpr, sub, rpb;
  __device__ RowMap()
      : t(WG ? threadIdx.x : threadIdx.x & 63), tpr(WG ? blockDim.x : 64), sub(WG ? 0 : threadIdx.x >> 6),
        rpb(WG ? 1 : 4) {}
};

// ------------------------------------------------------------ forward
template <bool WG, int VPT, int PASS, bool SR, bool XF, bool RF>
__global__ __launch_bounds__(WG ? 1024 : 256) void rmsnorm_fwd_kernel(NormFwd A) {
  constexpr bool QUANT = PASS == SNIP_FP8_E4M3 || PASS == SNIP_NVFP4 || PASS == SNIP_MXFP4;
  __shared__ float red[2][16];
  __shared__ uint32_t ured[32];
  __shared__ double dred[32];
  __shared__ float inv_lut[PASS == SNIP_NVFP4 ? 128 : 1];
  const RowMap<WG> R;
  const int t = R.t;
  const int64_t step = (int64_t)gridDim.x * R.rpb;
  int64_t row = (int64_t)blockIdx.x * R.rpb + R.sub;

  Raw<XF> rx[VPT] = {};
  Raw<RF> rr[VPT] = {};
  float g[VPT][8];
  auto load = [&](int64_t i) {
    if (i < A.rows) {
      load_row(A.x.p, i * A.x.ld, t, R.tpr, A.cols, rx);
      if (A.res.p) load_row(A.res.p, i * A.res.ld, t, R.tpr, A.cols, rr);
    }
  };
  load(row);
  load_gamma(A.gamma, t, R.tpr, A.cols, g);

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
    ss = row_sum<WG>(ss, red, it & 1);
    const float r = 1.0f / sqrtf(ss / (float)A.cols + A.eps);
    if constexpr (PASS != kPassAmax) {
      if (A.h.p) store_row(A.h, row, t, R.tpr, A.cols, h);
      if (A.rstd && t == 0) A.rstd[row] = r;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * r * g[v][i];
    if constexpr (PASS == kPassAmax) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (8 * (t + v * R.tpr) < A.cols) amax = chunk_max_bits(h[v], amax);
    } else {
      if (A.y.p) store_row(A.y, row, t, R.tpr, A.cols, h);
      if constexpr (QUANT) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
          if (t + v * R.tpr < qch) quant_chunk<PASS, SR>(A.q, eS, inv_lut, row * qch + t + v * R.tpr, h[v], stats, acc);
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
template <bool WG, int VPT, bool YF, bool HF, bool RF>
__global__ __launch_bounds__(WG ? 1024 : 256) void rmsnorm_bwd_kernel(NormBwd A) {
  __shared__ float red[2][16];
  __shared__ float lds[WG ? 1 : 3][WG ? 1 : VPT * 8 * 64];
  const RowMap<WG> R;
  const int t = R.t, sub = R.sub;
  const int64_t step = (int64_t)gridDim.x * R.rpb;
  int64_t row = (int64_t)blockIdx.x * R.rpb + sub;

  Raw<YF> ry[VPT] = {};
  Raw<HF> rh[VPT] = {};
  Raw<RF> rr[VPT] = {};
  float g[VPT][8];
  float rs = 0.0f;
  auto load = [&](int64_t i) {
    if (i < A.rows) {
      load_row(A.dy.p, i * A.dy.ld, t, R.tpr, A.cols, ry);
      load_row(A.h.p, i * A.h.ld, t, R.tpr, A.cols, rh);
      if (A.dres.p) load_row(A.dres.p, i * A.dres.ld, t, R.tpr, A.cols, rr);
      rs = A.rstd[i];
    }
  };
  load(row);
  load_gamma(A.gamma, t, R.tpr, A.cols, g);
  float dg[VPT][8];
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[v][i] = 0.0f;

  // the next row's loads run while this one is worked on, but with two chunks a
  // thread of 1024, whose 128 registers hardly hold one row: even so, of those
  // forms the ones with bf16 dy and fp32 h or fp32 dres, and the all-fp32 one,
  // spill 24 to 60 registers (36 to 52 bytes a lane)
  constexpr bool AHEAD = VPT == 1 || !WG;
  for (int it = 0; row < A.rows; ++it, row += step) {
    if (!AHEAD && it > 0) load(row);
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
    if (AHEAD) load(row + step);
    const float mean = row_sum<WG>(dot, red, it & 1) / (float)A.cols;
    if (A.dx.p) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[v][i] = r * fmaf(-xh[v][i], mean, d[v][i]);
          if (A.dres.p) d[v][i] += res[v][i];
        }
      store_row(A.dx, row, t, R.tpr, A.cols, d);
    }
  }
  if (!A.part) return;
  if constexpr (!WG) {
    if (sub > 0) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) lds[sub - 1][(v * 8 + i) * 64 + t] = dg[v][i];
    }
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[v][i] += lds[s][(v * 8 + i) * 64 + t];
  }
  float* dst = A.part + (int64_t)blockIdx.x * A.part_ld;
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    if (8 * (t + v * R.tpr) < A.part_ld) store_whole(dst, true, 8 * (t + v * R.tpr), dg[v]);
}

// dgamma[c] = sum over the workgroups' partial rows: 8 threads x 4 columns
// (a 128-byte line of a row), 32 slices of the rows joined through LDS.
__global__ __launch_bounds__(256) void dgamma_sum_kernel(const float* part, int64_t ld, int nwg, int cols,
                                                         float* dgamma) {
  __shared__ float red[32][33];
  const int cx = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int64_t c = ((int64_t)blockIdx.x * 8 + cx) * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < ld) {
#pragma unroll 8
    for (int i = slice; i < nwg; i += 32) {
      const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)i * ld + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  red[slice][4 * cx] = s.x;
  red[slice][4 * cx + 1] = s.y;
  red[slice][4 * cx + 2] = s.z;
  red[slice][4 * cx + 3] = s.w;
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && col < cols) {
    float v = red[0][threadIdx.x];
#pragma unroll
    for (int k = 1; k < 32; ++k) v += red[k][threadIdx.x];
    dgamma[col] = v;
  }
}

// ------------------------------------------------------------ statistics
// The statistics of a forward launch from its workgroups' partials, in a fixed
// order.
__global__ __launch_bounds__(256) void op_stats_kernel(const StatPart* part, int n, snip_stats* out) {
  __shared__ double dred[8];
  __shared__ uint32_t ured[8];
  StatPart p{0.0, 0.0, 0u, 0u};
#pragma unroll
  for (int j = 0; j < kOpsWG / 256; ++j) {
    const int i = threadIdx.x + 256 * j;
    if (i < n) {
      const StatPart o = part[i];
      p.e2 += o.e2;
      p.x2 += o.x2;
      p.nf += o.nf;
      p.amax_bits = max(p.amax_bits, o.amax_bits);
    }
  }
  const double e2 = wave_sum(p.e2), x2 = wave_sum(p.x2);
  const uint32_t nf = wave_sum_u(p.nf), am = wave_max_u(p.amax_bits);
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    dred[2 * wave] = e2;
    dred[2 * wave + 1] = x2;
    ured[2 * wave] = nf;
    ured[2 * wave + 1] = am;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    snip_stats s{0.0, 0.0, 0.0f, 0u};
    uint32_t m = 0u;
    for (int w = 0; w < 4; ++w) {
      s.sum_err2 += dred[2 * w];
      s.sum_x2 += dred[2 * w + 1];
      s.n_nonfinite += ured[2 * w];
      m = max(m, ured[2 * w + 1]);
    }
    s.amax = __uint_as_float(m);
    *out = s;
  }
}

hipError_t launch_op_stats(const StatPart* part, int n, snip_stats* out, hipStream_t s) {
  op_stats_kernel<<<dim3(1), dim3(256), 0, s>>>(part, n, out);
  return hipGetLastError();
}

// ------------------------------------------------------------ shapes
namespace {
struct NormShape {
  bool wg;        // a row to a workgroup
  int vpt, threads;
};

// A wave to a row up to 1024 columns, two chunks a lane beyond 512 (16384 x 640,
// fp32 residual: forward to bf16 and FP8 27.6 us, 33.0 as workgroups of 128;
// backward 24.6 and 36.6). Wider, a workgroup with a chunk a thread up to
// `one_up_to` chunks, two beyond. The forward pass takes two beyond 4096 columns
// (4096 x 8192 bf16 to FP8: 44.4 us, 46.4 with one and 1024 threads); the
// backward pass, with its column sums, is short of registers then and takes two
// where it must (4096 x 8192, fp32 residual: 67 us with one, 83 with two; 1003 x
// 4104: 14.1 and 16.3).
NormShape norm_shape(int64_t cols, int one_up_to) {
  const int64_t ch = ceil_div(cols, 8);
  if (ch <= 128) return {false, ch <= 64 ? 1 : 2, 256};
  const int vpt = ch <= one_up_to ? 1 : 2;
  return {true, vpt, (int)(64 * ceil_div(ch, 64 * vpt))};
}
NormShape fwd_shape(int64_t cols) { return norm_shape(cols, 512); }
NormShape bwd_shape(int64_t cols) { return norm_shape(cols, 1024); }

int norm_wg(const NormShape& k, int64_t rows, int most) {
  const int64_t n = k.wg ? rows : ceil_div(rows, 4);
  return (int)(n < most ? n : most);
}

// f(WG, VPT) as constants for the row's shape.
template <class F>
void with_shape(const NormShape& k, F f) {
  using one = std::integral_constant<int, 1>;
  using two = std::integral_constant<int, 2>;
  if (!k.wg) return k.vpt == 1 ? f(std::false_type{}, one{}) : f(std::false_type{}, two{});
  if (k.vpt == 1) return f(std::true_type{}, one{});
  return f(std::true_type{}, two{});
}

// f(F32) for a matrix's type; an absent one counts as bf16.
template <class F>
void with_type(const Mat& m, F f) {
  if (m.p && m.type == SNIPOP_F32) return f(std::true_type{});
  return f(std::false_type{});
}

template <int PASS, bool SR>
hipError_t norm_fwd_pass(const NormFwd& a, int nwg, hipStream_t s) {
  const NormShape k = fwd_shape(a.cols);
  with_shape(k, [&](auto wg, auto vpt) {
    with_type(a.x, [&](auto xf) {
      with_type(a.res, [&](auto rf) {
        rmsnorm_fwd_kernel<decltype(wg)::value, decltype(vpt)::value, PASS, SR, decltype(xf)::value,
                           decltype(rf)::value><<<dim3(nwg), dim3(k.threads), 0, s>>>(a);
      });
    });
  });
  return hipGetLastError();
}
template <int FMT>
hipError_t norm_fwd_quant(const NormFwd& a, int nwg, hipStream_t s) {
  return a.q.sr ? norm_fwd_pass<FMT, true>(a, nwg, s) : norm_fwd_pass<FMT, false>(a, nwg, s);
}
}  // namespace

// As many workgroups as are resident, 16 waves on each of the 256 CUs: a row's
// loads then run while the row before is worked on (fp32 residual, to FP8, 4096 x
// 4096: 30.2 us with 512 workgroups of 8 waves, 31.2 with 1024; 4096 x 2048:
// 18.0 us with 1024 of 4 waves, 21.2 with 512).
int norm_fwd_wg(int64_t rows, int64_t cols) {
  const NormShape k = fwd_shape(cols);
  const int per_cu = 1024 / k.threads;
  static_assert(256 * 4 <= kOpsWG, "one partial a workgroup, at most 4 workgroups a CU");
  return norm_wg(k, rows, 256 * (per_cu < 1 ? 1 : per_cu > 4 ? 4 : per_cu));
}
// Each workgroup leaves a partial row of dgamma, to be written and read
// again: as few as keep the card busy (1003 x 4104: 14 us with 256, 16 with
// 512; 4096 x 2048: 24 and 20).
int norm_bwd_wg(int64_t rows, int64_t cols) {
  const NormShape k = bwd_shape(cols);
  return norm_wg(k, rows, k.threads > 512 ? 256 : 512);
}

hipError_t launch_norm_fwd(int pass, const NormFwd& a, int nwg, hipStream_t s) {
  switch (pass) {
    case kPassAmax: return norm_fwd_pass<kPassAmax, false>(a, nwg, s);
    case SNIP_FP8_E4M3: return norm_fwd_quant<SNIP_FP8_E4M3>(a, nwg, s);
    case SNIP_NVFP4: return norm_fwd_quant<SNIP_NVFP4>(a, nwg, s);
    case SNIP_MXFP4: return norm_fwd_quant<SNIP_MXFP4>(a, nwg, s);
    default: return norm_fwd_pass<SNIP_BF16, false>(a, nwg, s);
  }
}

hipError_t launch_norm_bwd(const NormBwd& a, float* dgamma, int nwg, hipStream_t s) {
  const NormShape k = bwd_shape(a.cols);
  with_shape(k, [&](auto wg, auto vpt) {
    with_type(a.dy, [&](auto yf) {
      with_type(a.h, [&](auto hf) {
        with_type(a.dres, [&](auto rf) {
          rmsnorm_bwd_kernel<decltype(wg)::value, decltype(vpt)::value, decltype(yf)::value, decltype(hf)::value,
                             decltype(rf)::value><<<dim3(nwg), dim3(k.threads), 0, s>>>(a);
        });
      });
    });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dgamma) return e;
  dgamma_sum_kernel<<<dim3((unsigned)ceil_div(a.cols, 32)), dim3(256), 0, s>>>(a.part, a.part_ld, nwg, a.cols,
                                                                              dgamma);
  return hipGetLastError();
}

}  // namespace snip
