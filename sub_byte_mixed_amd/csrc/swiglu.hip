// SwiGLU, y = gate * sigmoid(gate) * up, forward (with an optional output
// quantized for the next GEMM) and backward, for gfx950.
//
// Elementwise scans, bound by HBM with the vector ALU not far behind. A
// thread takes chunks of E elements along the flattened [rows][ceil(cols / E)]
// grid of chunks, E being 16 bytes of gate (a wave's load is then one run of
// 1 KB: with two loads of every other 16 bytes, reads past the caches lose a
// fifth), so that neighbouring lanes hold neighbouring chunks of a
// row (the blocks of a quantized output need that); it advances by the grid's
// stride in rows and chunks that the host has divided once, and the next
// chunk's loads are issued before the present one is worked on. Measured:
// forward 8192 x 11008, fp32 to FP8, 142 us (5.7 TB/s), to NVFP4 149, to MX-FP4
// 146, with its own maximum 243 to FP8; backward 4096 x 5632, fp32 in, bf16 out,
// 58.8 us (6.3 TB/s: mostly reads, part of them cached).
#include "row_common.h"

namespace snip {

// A thread's walk over the grid of chunks.
struct Walk {
  int64_t row, at;             // row, and index in the grid of chunks
  int32_t ch;                  // chunk of the row
  bool wrapped;                // the last step went past the end of a row

  __device__ Walk(int32_t per_row) : at((int64_t)blockIdx.x * 256 + threadIdx.x), wrapped(false) {
    row = at / per_row;
    ch = (int32_t)(at % per_row);
  }
  __device__ void step(const GateStride& d, int32_t per_row) {
    at += (int64_t)gridDim.x * 256;
    row += d.rows;
    ch += d.chunks;
    wrapped = ch >= per_row;
    if (wrapped) {
      ch -= per_row;
      ++row;
    }
  }
};

// The element offset of the walk's chunk in one matrix, kept by additions.
template <int E>
struct Offset {
  int64_t off, step, wrap;
  __device__ Offset(const Mat& m, const Walk& w, const GateStride& d, int32_t per_row)
      : off(w.row * m.ld + E * (int64_t)w.ch), step(d.rows * m.ld + E * (int64_t)d.chunks),
        wrap(m.ld - E * (int64_t)per_row) {}
  __device__ void follow(const Walk& w) { off += step + (w.wrapped ? wrap : 0); }
};

// `tail`: cols % E, the elements of a row's last chunk (0: a whole one).
template <bool NT, bool F32, int E>
__device__ __forceinline__ void load_chunk(const Mat& m, const Offset<E>& o, bool last, int tail, Raw<F32, E>& r) {
  if (tail && last)
    load_partial(m.p, o.off, tail, r);
  else
    load_whole<NT>(m.p, o.off, r);
}
template <int E>
__device__ __forceinline__ void store_chunk(const Mat& m, const Offset<E>& o, bool last, int tail,
                                            const float (&x)[E]) {
  if (tail && last)
    store_partial(m.p, m.type == SNIPOP_F32, o.off, tail, x);
  else
    store_whole(m.p, m.type == SNIPOP_F32, o.off, x);
}

// 1 / (1 + exp(-g)) within 7 half-ulps (2 each of the hardware's exp2 and
// reciprocal, 3 of the products and the sum): -g log2(e) in two parts, the
// second one's share as a factor. Beyond +-150 exp2 is 0 or infinite, and the
// sigmoid 1 or 0. 9 operations; the library's expf and division, about half an
// ulp each, take 30 (8192 x 11008 fp32 to FP8, one after the other: 146 and 157
// us). An fp32 y can be an ulp further off for it; bf16 and quantized ones have
// coarser roundings.
__device__ __forceinline__ float sigmoid(float g) {
  const float t = __builtin_amdgcn_fmed3f(-g, -150.0f, 150.0f);
  const float hi = t * 1.44269502f;
  const float lo = fmaf(t, 1.92596303e-8f, fmaf(t, 1.44269502f, -hi));
  const float e = __builtin_amdgcn_exp2f(hi) * fmaf(lo, 0.693147182f, 1.0f);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

template <int PASS, bool SR, bool F32, bool NT>
__global__ __launch_bounds__(256) void swiglu_fwd_kernel(GateFwd A) {
  constexpr bool QUANT = PASS == SNIP_FP8_E4M3 || PASS == SNIP_NVFP4 || PASS == SNIP_MXFP4;
  __shared__ uint32_t ured[8];
  __shared__ double dred[8];
  __shared__ float inv_lut[PASS == SNIP_NVFP4 ? 128 : 1];
  constexpr int E = F32 ? 4 : 8;
  const int32_t per_row = (int32_t)((A.cols + E - 1) / E);
  const int tail = (int)(A.cols % E);
  Walk w(per_row);
  Offset<E> og(A.gate, w, A.d, per_row), ou(A.up, w, A.d, per_row), oy(A.y, w, A.d, per_row);
  Raw<F32, E> rg = {}, ru = {};
  auto load = [&]() {
    if (w.row < A.rows) {
      load_chunk<NT>(A.gate, og, w.ch == per_row - 1, tail, rg);
      load_chunk<NT>(A.up, ou, w.ch == per_row - 1, tail, ru);
    }
  };
  load();
  const int eS = QUANT ? op_tensor_exp<PASS>(A.q, ured) : 0;
  if constexpr (PASS == SNIP_NVFP4) fill_inv_lut(inv_lut);
  const bool stats = QUANT && A.q.part != nullptr;
  QAcc acc;
  uint32_t amax = 0u;
  while (w.row < A.rows) {
    float g[E], u[E];
    raw_to_f32(rg, g);
    raw_to_f32(ru, u);
    const bool last = w.ch == per_row - 1;
    const int64_t at = w.at;
    w.step(A.d, per_row);
    og.follow(w);
    ou.follow(w);
    load();
#pragma unroll
    for (int i = 0; i < E; ++i) g[i] = g[i] * sigmoid(g[i]) * u[i];
    if constexpr (PASS == kPassAmax) {
      amax = chunk_max_bits(g, amax);
    } else {
      if (A.y.p) store_chunk(A.y, oy, last, tail, g);
      oy.follow(w);
      if constexpr (QUANT) quant_chunk<PASS, SR>(A.q, eS, inv_lut, at, g, stats, acc);
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

// dgate = dy u s (1 + g (1 - s)), dup = dy g s: every input once, both
// outputs once.
template <bool YF, bool F32, bool NT>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(GateBwd A) {
  constexpr int E = F32 ? 4 : 8;
  const int32_t per_row = (int32_t)((A.cols + E - 1) / E);
  const int tail = (int)(A.cols % E);
  Walk w(per_row);
  Offset<E> od(A.dy, w, A.d, per_row), og(A.gate, w, A.d, per_row), ou(A.up, w, A.d, per_row);
  Offset<E> oa(A.dgate, w, A.d, per_row), ob(A.dup, w, A.d, per_row);
  Raw<YF, E> ry = {};
  Raw<F32, E> rg = {}, ru = {};
  auto load = [&]() {
    if (w.row < A.rows) {
      const bool last = w.ch == per_row - 1;
      load_chunk<NT>(A.dy, od, last, tail, ry);
      load_chunk<NT>(A.gate, og, last, tail, rg);
      load_chunk<NT>(A.up, ou, last, tail, ru);
    }
  };
  load();
  while (w.row < A.rows) {
    float d[E], g[E], u[E];
    raw_to_f32(ry, d);
    raw_to_f32(rg, g);
    raw_to_f32(ru, u);
    const bool last = w.ch == per_row - 1;
    w.step(A.d, per_row);
    od.follow(w);
    og.follow(w);
    ou.follow(w);
    load();
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float s = sigmoid(g[i]);
      const float gs = g[i] * s;
      u[i] = d[i] * u[i] * (s + gs * (1.0f - s));
      g[i] = d[i] * gs;
    }
    if (A.dgate.p) store_chunk(A.dgate, oa, last, tail, u);
    if (A.dup.p) store_chunk(A.dup, ob, last, tail, g);
    oa.follow(w);
    ob.follow(w);
  }
}

namespace {
int64_t chunks_per_row(const Mat& gate, int64_t cols) { return ceil_div(cols, gate.type == SNIPOP_F32 ? 4 : 8); }

GateStride stride_of(int nwg, const Mat& gate, int64_t cols) {
  const int64_t stride = (int64_t)nwg * 256, per_row = chunks_per_row(gate, cols);
  return GateStride{stride / per_row, (int32_t)(stride % per_row)};
}

// Inputs beyond the last-level cache (256 MB) are read past the caches:
// 4096 x 5632 backward, 369 MB: 71 -> 68 us; smaller ones may still lie there
// from the GEMM that wrote them.
bool beyond_cache(int64_t rows, int64_t cols, int bytes) {
  return (double)rows * (double)cols * bytes > 256.0 * 1024 * 1024;
}

int elem(const Mat& m) { return m.type == SNIPOP_F32 ? 4 : 2; }

template <int PASS, bool SR>
hipError_t gate_fwd_pass(const GateFwd& a, int nwg, hipStream_t s) {
  const dim3 grid(nwg), block(256);
  const bool nt = beyond_cache(a.rows, a.cols, 2 * elem(a.gate));
  if (a.gate.type == SNIPOP_F32) {
    if (nt)
      swiglu_fwd_kernel<PASS, SR, true, true><<<grid, block, 0, s>>>(a);
    else
      swiglu_fwd_kernel<PASS, SR, true, false><<<grid, block, 0, s>>>(a);
  } else {
    if (nt)
      swiglu_fwd_kernel<PASS, SR, false, true><<<grid, block, 0, s>>>(a);
    else
      swiglu_fwd_kernel<PASS, SR, false, false><<<grid, block, 0, s>>>(a);
  }
  return hipGetLastError();
}
template <int FMT>
hipError_t gate_fwd_quant(const GateFwd& a, int nwg, hipStream_t s) {
  return a.q.sr ? gate_fwd_pass<FMT, true>(a, nwg, s) : gate_fwd_pass<FMT, false>(a, nwg, s);
}

template <bool NT>
void gate_bwd_pass(const GateBwd& a, int nwg, hipStream_t s) {
  const dim3 grid(nwg), block(256);
  const bool yf = a.dy.type == SNIPOP_F32, f = a.gate.type == SNIPOP_F32;
  if (yf && f)
    swiglu_bwd_kernel<true, true, NT><<<grid, block, 0, s>>>(a);
  else if (yf)
    swiglu_bwd_kernel<true, false, NT><<<grid, block, 0, s>>>(a);
  else if (f)
    swiglu_bwd_kernel<false, true, NT><<<grid, block, 0, s>>>(a);
  else
    swiglu_bwd_kernel<false, false, NT><<<grid, block, 0, s>>>(a);
}
}  // namespace

int gate_wg(const Mat& gate, int64_t rows, int64_t cols, int most) {
  const int64_t wg = ceil_div(rows * chunks_per_row(gate, cols), 256);
  return (int)(wg < most ? wg : most);
}

hipError_t launch_gate_fwd(int pass, GateFwd a, int nwg, hipStream_t s) {
  a.d = stride_of(nwg, a.gate, a.cols);
  switch (pass) {
    case kPassAmax: return gate_fwd_pass<kPassAmax, false>(a, nwg, s);
    case SNIP_FP8_E4M3: return gate_fwd_quant<SNIP_FP8_E4M3>(a, nwg, s);
    case SNIP_NVFP4: return gate_fwd_quant<SNIP_NVFP4>(a, nwg, s);
    case SNIP_MXFP4: return gate_fwd_quant<SNIP_MXFP4>(a, nwg, s);
    default: return gate_fwd_pass<SNIP_BF16, false>(a, nwg, s);
  }
}

hipError_t launch_gate_bwd(GateBwd a, int nwg, hipStream_t s) {
  a.d = stride_of(nwg, a.gate, a.cols);
  if (beyond_cache(a.rows, a.cols, 2 * elem(a.gate) + elem(a.dy)))
    gate_bwd_pass<true>(a, nwg, s);
  else
    gate_bwd_pass<false>(a, nwg, s);
  return hipGetLastError();
}

}  // namespace snip
