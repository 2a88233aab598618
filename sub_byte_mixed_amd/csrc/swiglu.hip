// SwiGLU, y = gate * sigmoid(gate) * up, forward (with an optional output
// quantized for the next GEMM) and backward, for gfx950.
//
// Elementwise scans bound by HBM. A thread takes chunks of 8 elements along
// the flattened [rows][ceil(cols / 8)] grid of chunks, so that neighbouring
// lanes hold neighbouring chunks of a row (the blocks of a quantized output
// need that); it advances by the grid's stride in rows and chunks that the
// host has divided once, and the next chunk's loads are issued before the
// present one is worked on. sigmoid is 1 / (1 + exp(-g)) with the accurate
// exp and division of fp32: they cost less than the chunk's bytes.
#include "row_common.h"

namespace snip {

// A position in the grid of chunks.
struct ChunkPos {
  int64_t row, ch;
};

__device__ __forceinline__ ChunkPos first_chunk(int64_t per_row) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  return ChunkPos{i / per_row, i % per_row};
}
__device__ __forceinline__ ChunkPos next_chunk(const ChunkPos& p, int64_t drow, int64_t dchunk, int64_t per_row) {
  ChunkPos n{p.row + drow, p.ch + dchunk};
  if (n.ch >= per_row) {
    n.ch -= per_row;
    ++n.row;
  }
  return n;
}

template <bool F32>
__device__ __forceinline__ void load_chunk(const Mat& m, const ChunkPos& p, int64_t cols, Raw8<F32>& r) {
  const int64_t off = p.row * m.ld + 8 * p.ch;
  if (8 * p.ch + 8 <= cols)
    load_whole(m.p, off, r);
  else
    load_partial(m.p, off, (int)(cols - 8 * p.ch), r);
}
__device__ __forceinline__ void store_chunk(const Mat& m, const ChunkPos& p, int64_t cols, const float (&x)[8]) {
  const int64_t off = p.row * m.ld + 8 * p.ch;
  if (8 * p.ch + 8 <= cols)
    store_whole(m.p, m.type == SNIPOP_F32, off, x);
  else
    store_partial(m.p, m.type == SNIPOP_F32, off, (int)(cols - 8 * p.ch), x);
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

template <int PASS, bool F32>
__global__ __launch_bounds__(256) void swiglu_fwd_kernel(GateFwd A) {
  constexpr bool QUANT = PASS == SNIP_FP8_E4M3 || PASS == SNIP_NVFP4 || PASS == SNIP_MXFP4;
  __shared__ uint32_t ured[8];
  __shared__ double dred[8];
  __shared__ float inv_lut[PASS == SNIP_NVFP4 ? 128 : 1];
  const int64_t per_row = (A.cols + 7) >> 3;
  ChunkPos p = first_chunk(per_row);
  Raw8<F32> rg = {}, ru = {};
  auto load = [&](const ChunkPos& q) {
    if (q.row < A.rows) {
      load_chunk(A.gate, q, A.cols, rg);
      load_chunk(A.up, q, A.cols, ru);
    }
  };
  load(p);
  const int eS = QUANT ? op_tensor_exp<PASS>(A.q, ured) : 0;
  if constexpr (PASS == SNIP_NVFP4) fill_inv_lut(inv_lut);
  const bool stats = QUANT && A.q.part != nullptr;
  QAcc acc;
  uint32_t amax = 0u;
  while (p.row < A.rows) {
    float g[8], u[8];
    raw_to_f32(rg, g);
    raw_to_f32(ru, u);
    const ChunkPos n = next_chunk(p, A.drow, A.dchunk, per_row);
    load(n);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = g[i] * sigmoid(g[i]) * u[i];
    if constexpr (PASS == kPassAmax) {
      amax = chunk_max_bits(g, amax);
    } else {
      if (A.y.p) store_chunk(A.y, p, A.cols, g);
      if constexpr (QUANT) quant_chunk<PASS>(A.q, eS, inv_lut, p.row * per_row + p.ch, g, stats, acc);
    }
    p = n;
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
template <bool YF, bool F32>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(GateBwd A) {
  const int64_t per_row = (A.cols + 7) >> 3;
  ChunkPos p = first_chunk(per_row);
  Raw8<YF> ry = {};
  Raw8<F32> rg = {}, ru = {};
  auto load = [&](const ChunkPos& q) {
    if (q.row < A.rows) {
      load_chunk(A.dy, q, A.cols, ry);
      load_chunk(A.gate, q, A.cols, rg);
      load_chunk(A.up, q, A.cols, ru);
    }
  };
  load(p);
  while (p.row < A.rows) {
    float d[8], g[8], u[8];
    raw_to_f32(ry, d);
    raw_to_f32(rg, g);
    raw_to_f32(ru, u);
    const ChunkPos n = next_chunk(p, A.drow, A.dchunk, per_row);
    load(n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(g[i]);
      const float gs = g[i] * s;
      u[i] = d[i] * u[i] * (s + gs * (1.0f - s));
      g[i] = d[i] * gs;
    }
    if (A.dgate.p) store_chunk(A.dgate, p, A.cols, u);
    if (A.dup.p) store_chunk(A.dup, p, A.cols, g);
    p = n;
  }
}

namespace {
int64_t chunks_per_row(int64_t cols) { return ceil_div(cols, 8); }

template <int PASS>
hipError_t gate_fwd_pass(const GateFwd& a, int nwg, hipStream_t s) {
  if (a.gate.type == SNIPOP_F32)
    swiglu_fwd_kernel<PASS, true><<<dim3(nwg), dim3(256), 0, s>>>(a);
  else
    swiglu_fwd_kernel<PASS, false><<<dim3(nwg), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}
}  // namespace

int gate_wg(int64_t rows, int64_t cols, bool amax) {
  const int64_t wg = ceil_div(rows * chunks_per_row(cols), 256);
  const int most = amax ? kOpsAmaxWG : kOpsWG;
  return (int)(wg < most ? wg : most);
}

hipError_t launch_gate_fwd(int pass, GateFwd a, int nwg, hipStream_t s) {
  const int64_t stride = (int64_t)nwg * 256, per_row = chunks_per_row(a.cols);
  a.drow = stride / per_row;
  a.dchunk = stride % per_row;
  switch (pass) {
    case kPassAmax: return gate_fwd_pass<kPassAmax>(a, nwg, s);
    case SNIP_FP8_E4M3: return gate_fwd_pass<SNIP_FP8_E4M3>(a, nwg, s);
    case SNIP_NVFP4: return gate_fwd_pass<SNIP_NVFP4>(a, nwg, s);
    case SNIP_MXFP4: return gate_fwd_pass<SNIP_MXFP4>(a, nwg, s);
    default: return gate_fwd_pass<SNIP_BF16>(a, nwg, s);
  }
}

hipError_t launch_gate_bwd(GateBwd a, int nwg, hipStream_t s) {
  const int64_t stride = (int64_t)nwg * 256, per_row = chunks_per_row(a.cols);
  a.drow = stride / per_row;
  a.dchunk = stride % per_row;
  const dim3 grid(nwg), block(256);
  const bool yf = a.dy.type == SNIPOP_F32, f = a.gate.type == SNIPOP_F32;
  if (yf && f)
    swiglu_bwd_kernel<true, true><<<grid, block, 0, s>>>(a);
  else if (yf)
    swiglu_bwd_kernel<true, false><<<grid, block, 0, s>>>(a);
  else if (f)
    swiglu_bwd_kernel<false, true><<<grid, block, 0, s>>>(a);
  else
    swiglu_bwd_kernel<false, false><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace snip
