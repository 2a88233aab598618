// Internal launch interface between ops_api.hip and the kernels of the
// operators around the linear layers (rmsnorm.hip, swiglu.hip, qgemv.hip).
#pragma once

#include "../../include/snip_ops.h"
#include "kernels.h"

namespace snip {

// Most workgroups of a pass that leaves a partial each: the maximum's, and the
// statistics' (norm 4096 x 2048 to FP8: 18.0 us with 1024, 18.3 with 2048, and
// the launch that sums the partials is the shorter for it).
constexpr int kOpsWG = 1024;
// SwiGLU without statistics: workgroups that come and go spread better than a
// few that walk far (4096 x 5632 backward: 60 us with 32768, 67 with 1024).
constexpr int kGateWG = 32768;

// A matrix argument: rows of `ld` elements of `type` (SNIPOP_BF16 / _F32).
struct Mat {
  void* p;
  int64_t ld;
  int32_t type;
};

// Output quantization of a forward operator. `amax_part`: fp32 magnitude
// bits, one per workgroup of the pass for the maximum.
struct OpQuant {
  uint8_t* codes;
  uint8_t* scales;
  int32_t* texp;               // tensor exponent out or null
  const float* amax_in;        // supplied max or null
  const uint32_t* amax_part;
  int32_t n_amax_part;
  StatPart* part;              // [workgroups] or null (no statistics)
  uint64_t seed;
  uint32_t tensor_id;
  int32_t sr;
};

struct NormFwd {
  Mat x, res, gamma, h, y;     // p null: absent
  float* rstd;
  int64_t rows;
  int32_t cols;
  float eps;
  OpQuant q;
  uint32_t* amax_out;          // pass for the maximum: [workgroups]
};

struct NormBwd {
  Mat dy, h, gamma, dres, dx;
  const float* rstd;
  float* part;                 // dgamma partials [nwg][part_ld] or null
  int64_t part_ld;
  int64_t rows;
  int32_t cols;
};

// A grid's stride over the chunks of a matrix, in rows and chunks.
struct GateStride {
  int64_t rows;
  int32_t chunks;
};

struct GateFwd {
  Mat gate, up, y;
  int64_t rows, cols;
  GateStride d;
  OpQuant q;
  uint32_t* amax_out;
};

struct GateBwd {
  Mat dy, gate, up, dgate, dup;
  int64_t rows, cols;
  GateStride d;
};

struct Gemv {
  const uint16_t* x;
  const uint8_t* codes;
  const uint8_t* scales;
  const int32_t* texp;
  void* y;
  int64_t ldx, ldy, N, K;
  int32_t M, y_type;
};

// What a forward launch leaves behind: SNIP_BF16 = y / h only, FP8, NVFP4,
// MXFP4 = codes too, kPassAmax = the maximum of |y| alone.
constexpr int kPassAmax = -1;

// Grids, and asynchronous launchers that return the launch's hipError_t.
int norm_fwd_wg(int64_t rows, int64_t cols);
int norm_bwd_wg(int64_t rows, int64_t cols);
int gate_wg(const Mat& gate, int64_t rows, int64_t cols, int most);
hipError_t launch_norm_fwd(int pass, const NormFwd& a, int nwg, hipStream_t s);
hipError_t launch_norm_bwd(const NormBwd& a, float* dgamma, int nwg, hipStream_t s);
hipError_t launch_gate_fwd(int pass, GateFwd a, int nwg, hipStream_t s);
hipError_t launch_gate_bwd(GateBwd a, int nwg, hipStream_t s);
hipError_t launch_op_stats(const StatPart* part, int n, snip_stats* out, hipStream_t s);
hipError_t launch_gemv(int format, const Gemv& a, hipStream_t s);

}  // namespace snip
