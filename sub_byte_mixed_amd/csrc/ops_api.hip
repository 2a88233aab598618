// Host side of include/snip_ops.h: argument validation (before any HIP
// call), workspace carving and kernel enqueueing for the operators around
// the quantized linear layers.
#include <cmath>
#include <cstring>

#include "api_common.h"
#include "ops.h"

using namespace snip;

namespace {

// Rows, leading dimensions and elements of a matrix: 64-bit byte offsets.
constexpr int64_t kMaxDim = (int64_t)1 << 40;
constexpr double kMaxElems = 1152921504606846976.0;   // 2^60
constexpr int64_t kMaxGateCols = (int64_t)1 << 31;   // a row's chunks are counted in 32 bits

// Scratch of a quantized output: partials of the pass for the maximum, and
// of the statistics.
constexpr size_t kOpsAmaxBytes = align_up(kOpsWG * sizeof(uint32_t), kAlign);
constexpr size_t kOpsQuantWS = kOpsAmaxBytes + align_up(kOpsWG * sizeof(StatPart), kAlign);

bool out_format(int f) { return f == SNIP_FP8_E4M3 || f == SNIP_NVFP4 || f == SNIP_MXFP4; }

int check_type(const char* who, const char* name, int type) {
  if (type != SNIPOP_BF16 && type != SNIPOP_F32)
    return fail(SNIP_E_FORMAT, "%s: %s: unknown element type %d", who, name, type);
  return SNIP_OK;
}

// A matrix argument that may be absent (p NULL), into `m`.
int check_mat(const char* who, const char* name, const void* p, int type, int64_t ld, int64_t rows, int64_t cols,
              Mat* m) {
  *m = Mat{nullptr, 0, SNIPOP_BF16};
  if (!p) return SNIP_OK;
  int rc = check_type(who, name, type);
  if (rc) return rc;
  if (ld < cols || ld > kMaxDim || ld % (type == SNIPOP_F32 ? 4 : 8))
    return fail(SNIP_E_SHAPE, "%s: %s: leading dimension %lld must be >= %lld and a multiple of %d", who, name,
                (long long)ld, (long long)cols, type == SNIPOP_F32 ? 4 : 8);
  if ((double)rows * (double)ld > kMaxElems)
    return fail(SNIP_E_SHAPE, "%s: %s: %lld rows of %lld elements are too many", who, name, (long long)rows,
                (long long)ld);
  if (!aligned(p, 16)) return fail(SNIP_E_ALIGN, "%s: %s is not 16-byte aligned", who, name);
  *m = Mat{const_cast<void*>(p), ld, type};
  return SNIP_OK;
}

// Shapes that the calls take.
bool valid_shape(int64_t rows, int64_t cols, int64_t max_cols) {
  return rows > 0 && rows <= kMaxDim && cols > 0 && cols <= max_cols;
}

int check_shape(const char* who, int64_t rows, int64_t cols, int64_t max_cols) {
  if (rows <= 0 || rows > kMaxDim || cols <= 0)
    return fail(SNIP_E_SHAPE, "%s: rows=%lld cols=%lld must be > 0", who, (long long)rows, (long long)cols);
  if (cols > max_cols)
    return fail(SNIP_E_SHAPE, "%s: cols=%lld above the limit of %lld", who, (long long)cols, (long long)max_cols);
  return SNIP_OK;
}

// The quantized output of a forward operator, checked and carved: q for the
// kernels, *amax for the pass for the maximum (NULL where none is needed).
int check_out(const char* who, const snip_qtensor* out, int64_t rows, int64_t cols, int rounding, uint64_t seed,
              uint32_t tensor_id, const float* amax_in, snip_stats* stats, void* ws, size_t ws_bytes, OpQuant* q,
              uint32_t** amax) {
  std::memset(q, 0, sizeof(*q));
  *amax = nullptr;
  if (!out) {
    if (stats) return fail(SNIP_E_NULL, "%s: statistics need a quantized output", who);
    return SNIP_OK;
  }
  int rc = validate_qtensor(out, who);
  if (rc) return rc;
  if (!out_format(out->format))
    return fail(SNIP_E_FORMAT, "%s: output format %d is not FP8_E4M3, NVFP4 or MXFP4", who, out->format);
  if (rounding != SNIP_RNE && rounding != SNIP_SR) return fail(SNIP_E_FORMAT, "%s: unknown rounding %d", who, rounding);
  if (cols % block_of(out->format))
    return fail(SNIP_E_SHAPE, "%s: cols=%lld not a multiple of %d", who, (long long)cols, block_of(out->format));
  if (out->rows != rows || out->k != cols)
    return fail(SNIP_E_SHAPE, "%s: out is [%lld][%lld], expected [%lld][%lld]", who, (long long)out->rows,
                (long long)out->k, (long long)rows, (long long)cols);
  if (!aligned(amax_in, 4) || !aligned(stats, 8) || !aligned(ws, 16))
    return fail(SNIP_E_ALIGN, "%s: misaligned pointer", who);
  const bool find = needs_amax(out->format) && !amax_in;
  if ((find || stats) && (!ws || ws_bytes < kOpsQuantWS))
    return fail(SNIP_E_WORKSPACE, "%s: workspace of %zu bytes needed", who, kOpsQuantWS);
  Carver cv(ws);
  uint32_t* ap = find ? reinterpret_cast<uint32_t*>(cv.take(kOpsAmaxBytes)) : nullptr;
  StatPart* sp = stats ? reinterpret_cast<StatPart*>(cv.take(kOpsWG * sizeof(StatPart))) : nullptr;
  *amax = ap;
  q->codes = static_cast<uint8_t*>(out->codes);
  q->scales = static_cast<uint8_t*>(out->scales);
  q->texp = has_texp(out->format) ? out->tensor_exp : nullptr;
  q->amax_in = amax_in;
  q->amax_part = ap;
  q->part = sp;
  q->seed = seed;
  q->tensor_id = tensor_id;
  q->sr = rounding == SNIP_SR;
  return SNIP_OK;
}

int finalize(const OpQuant& q, int nwg, snip_stats* stats, hipStream_t s) {
  if (!stats) return SNIP_OK;
  const int slot = timing_begin(LaunchTag{SNIP_LAUNCH_FINALIZE, -1, -1, -1, 1.0}, s);
  const hipError_t e = launch_op_stats(q.part, nwg, stats, s);
  timing_end(slot, s);
  return hip_check(e, "finalize launch");
}

LaunchTag op_tag(int kind, const snip_qtensor* out, int rounding, double work) {
  return LaunchTag{kind, out ? out->format : -1, out ? SNIP_ROWWISE : -1, out ? rounding : -1, work};
}

}  // namespace

extern "C" {

size_t snipop_rmsnorm_fwd_workspace(int64_t rows, int64_t cols, int format) {
  if (!valid_shape(rows, cols, SNIPOP_NORM_MAX_COLS) || !out_format(format) || cols % block_of(format)) return 0;
  return kOpsQuantWS;
}

size_t snipop_swiglu_fwd_workspace(int64_t rows, int64_t cols, int format) {
  if (!valid_shape(rows, cols, kMaxGateCols) || !out_format(format) || cols % block_of(format)) return 0;
  return kOpsQuantWS;
}

size_t snipop_rmsnorm_bwd_workspace(int64_t rows, int64_t cols) {
  if (!valid_shape(rows, cols, SNIPOP_NORM_MAX_COLS)) return 0;
  return align_up((size_t)norm_bwd_wg(rows, cols) * align_up((size_t)cols, 8) * sizeof(float), kAlign);
}

int snipop_rmsnorm_fwd(const void* x, int x_type, int64_t ldx, const void* res, int res_type, int64_t ldr,
                       const void* gamma, int gamma_type, int64_t rows, int64_t cols, float eps, void* h, int h_type,
                       int64_t ldh, void* y, int y_type, int64_t ldy, float* rstd, const snip_qtensor* out,
                       int rounding, uint64_t seed, uint32_t tensor_id, const float* amax_in, snip_stats* stats,
                       void* ws, size_t ws_bytes, void* stream) {
  const char* who = "snipop_rmsnorm_fwd";
  if (!x || !gamma) return fail(SNIP_E_NULL, "%s: x and gamma must be non-NULL", who);
  if (!h && !y && !rstd && !out) return fail(SNIP_E_NULL, "%s: no output given", who);
  int rc = check_shape(who, rows, cols, SNIPOP_NORM_MAX_COLS);
  if (rc) return rc;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(SNIP_E_SHAPE, "%s: eps must be finite and >= 0", who);
  NormFwd a;
  std::memset(&a, 0, sizeof(a));
  if ((rc = check_mat(who, "x", x, x_type, ldx, rows, cols, &a.x))) return rc;
  if ((rc = check_mat(who, "res", res, res_type, ldr, rows, cols, &a.res))) return rc;
  if ((rc = check_mat(who, "h", h, h_type, ldh, rows, cols, &a.h))) return rc;
  if ((rc = check_mat(who, "y", y, y_type, ldy, rows, cols, &a.y))) return rc;
  if ((rc = check_type(who, "gamma", gamma_type))) return rc;
  if (!aligned(gamma, 16) || !aligned(rstd, 4)) return fail(SNIP_E_ALIGN, "%s: misaligned pointer", who);
  a.gamma = Mat{const_cast<void*>(gamma), 0, gamma_type};
  uint32_t* amax;
  if ((rc = check_out(who, out, rows, cols, rounding, seed, tensor_id, amax_in, stats, ws, ws_bytes, &a.q, &amax)))
    return rc;
  a.rstd = rstd;
  a.rows = rows;
  a.cols = (int32_t)cols;
  a.eps = eps;

  hipStream_t s = static_cast<hipStream_t>(stream);
  const double work = (double)rows * (double)cols;
  if (amax) {
    a.amax_out = amax;
    a.q.n_amax_part = norm_fwd_wg(rows, cols);
    const int slot = timing_begin(LaunchTag{SNIP_LAUNCH_AMAX, -1, -1, -1, work}, s);
    const hipError_t e = launch_norm_fwd(kPassAmax, a, a.q.n_amax_part, s);
    timing_end(slot, s);
    if ((rc = hip_check(e, "norm amax launch"))) return rc;
  }
  const int nwg = norm_fwd_wg(rows, cols);
  const int slot = timing_begin(op_tag(SNIPOP_LAUNCH_NORM, out, rounding, work), s);
  const hipError_t e = launch_norm_fwd(out ? out->format : SNIP_BF16, a, nwg, s);
  timing_end(slot, s);
  if ((rc = hip_check(e, "norm launch"))) return rc;
  if ((rc = finalize(a.q, nwg, stats, s))) return rc;
  return ok();
}

int snipop_rmsnorm_bwd(const void* dy, int dy_type, int64_t lddy, const void* h, int h_type, int64_t ldh,
                       const void* gamma, int gamma_type, const float* rstd, const void* dres, int dres_type,
                       int64_t lddres, int64_t rows, int64_t cols, void* dx, int dx_type, int64_t lddx,
                       float* dgamma, void* ws, size_t ws_bytes, void* stream) {
  const char* who = "snipop_rmsnorm_bwd";
  if (!dy || !h || !gamma || !rstd) return fail(SNIP_E_NULL, "%s: dy, h, gamma and rstd must be non-NULL", who);
  if (!dx && !dgamma) return fail(SNIP_E_NULL, "%s: no output given", who);
  int rc = check_shape(who, rows, cols, SNIPOP_NORM_MAX_COLS);
  if (rc) return rc;
  NormBwd a;
  std::memset(&a, 0, sizeof(a));
  if ((rc = check_mat(who, "dy", dy, dy_type, lddy, rows, cols, &a.dy))) return rc;
  if ((rc = check_mat(who, "h", h, h_type, ldh, rows, cols, &a.h))) return rc;
  if ((rc = check_mat(who, "dres", dres, dres_type, lddres, rows, cols, &a.dres))) return rc;
  if ((rc = check_mat(who, "dx", dx, dx_type, lddx, rows, cols, &a.dx))) return rc;
  if ((rc = check_type(who, "gamma", gamma_type))) return rc;
  if (!aligned(gamma, 16) || !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(ws, 16))
    return fail(SNIP_E_ALIGN, "%s: misaligned pointer", who);
  const size_t need = snipop_rmsnorm_bwd_workspace(rows, cols);
  if (dgamma && (!ws || ws_bytes < need)) return fail(SNIP_E_WORKSPACE, "%s: workspace of %zu bytes needed", who, need);
  a.gamma = Mat{const_cast<void*>(gamma), 0, gamma_type};
  a.rstd = rstd;
  a.part = dgamma ? static_cast<float*>(ws) : nullptr;
  a.part_ld = (int64_t)align_up((size_t)cols, 8);
  a.rows = rows;
  a.cols = (int32_t)cols;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int slot = timing_begin(op_tag(SNIPOP_LAUNCH_NORM, nullptr, -1, (double)rows * (double)cols), s);
  const hipError_t e = launch_norm_bwd(a, dgamma, norm_bwd_wg(rows, cols), s);
  timing_end(slot, s);
  if ((rc = hip_check(e, "norm backward launch"))) return rc;
  return ok();
}

int snipop_swiglu_fwd(const void* gate, int64_t ldg, const void* up, int64_t ldu, int type, int64_t rows,
                      int64_t cols, void* y, int y_type, int64_t ldy, const snip_qtensor* out, int rounding,
                      uint64_t seed, uint32_t tensor_id, const float* amax_in, snip_stats* stats, void* ws,
                      size_t ws_bytes, void* stream) {
  const char* who = "snipop_swiglu_fwd";
  if (!gate || !up) return fail(SNIP_E_NULL, "%s: gate and up must be non-NULL", who);
  if (!y && !out) return fail(SNIP_E_NULL, "%s: no output given", who);
  int rc = check_shape(who, rows, cols, kMaxGateCols);
  if (rc) return rc;
  GateFwd a;
  std::memset(&a, 0, sizeof(a));
  if ((rc = check_mat(who, "gate", gate, type, ldg, rows, cols, &a.gate))) return rc;
  if ((rc = check_mat(who, "up", up, type, ldu, rows, cols, &a.up))) return rc;
  if ((rc = check_mat(who, "y", y, y_type, ldy, rows, cols, &a.y))) return rc;
  uint32_t* amax;
  if ((rc = check_out(who, out, rows, cols, rounding, seed, tensor_id, amax_in, stats, ws, ws_bytes, &a.q, &amax)))
    return rc;
  a.rows = rows;
  a.cols = cols;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const double work = (double)rows * (double)cols;
  if (amax) {
    a.amax_out = amax;
    a.q.n_amax_part = gate_wg(a.gate, rows, cols, kOpsWG);
    const int slot = timing_begin(LaunchTag{SNIP_LAUNCH_AMAX, -1, -1, -1, work}, s);
    const hipError_t e = launch_gate_fwd(kPassAmax, a, a.q.n_amax_part, s);
    timing_end(slot, s);
    if ((rc = hip_check(e, "swiglu amax launch"))) return rc;
  }
  const int nwg = gate_wg(a.gate, rows, cols, stats ? kOpsWG : kGateWG);
  const int slot = timing_begin(op_tag(SNIPOP_LAUNCH_GATE, out, rounding, work), s);
  const hipError_t e = launch_gate_fwd(out ? out->format : SNIP_BF16, a, nwg, s);
  timing_end(slot, s);
  if ((rc = hip_check(e, "swiglu launch"))) return rc;
  if ((rc = finalize(a.q, nwg, stats, s))) return rc;
  return ok();
}

int snipop_swiglu_bwd(const void* dy, int dy_type, int64_t lddy, const void* gate, int64_t ldg, const void* up,
                      int64_t ldu, int type, int64_t rows, int64_t cols, void* dgate, int64_t lddg, void* dup,
                      int64_t lddu, int d_type, void* stream) {
  const char* who = "snipop_swiglu_bwd";
  if (!dy || !gate || !up) return fail(SNIP_E_NULL, "%s: dy, gate and up must be non-NULL", who);
  if (!dgate && !dup) return fail(SNIP_E_NULL, "%s: no output given", who);
  int rc = check_shape(who, rows, cols, kMaxGateCols);
  if (rc) return rc;
  GateBwd a;
  std::memset(&a, 0, sizeof(a));
  if ((rc = check_mat(who, "dy", dy, dy_type, lddy, rows, cols, &a.dy))) return rc;
  if ((rc = check_mat(who, "gate", gate, type, ldg, rows, cols, &a.gate))) return rc;
  if ((rc = check_mat(who, "up", up, type, ldu, rows, cols, &a.up))) return rc;
  if ((rc = check_mat(who, "dgate", dgate, d_type, lddg, rows, cols, &a.dgate))) return rc;
  if ((rc = check_mat(who, "dup", dup, d_type, lddu, rows, cols, &a.dup))) return rc;
  a.rows = rows;
  a.cols = cols;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int slot = timing_begin(op_tag(SNIPOP_LAUNCH_GATE, nullptr, -1, (double)rows * (double)cols), s);
  const hipError_t e = launch_gate_bwd(a, gate_wg(a.gate, rows, cols, kGateWG), s);
  timing_end(slot, s);
  if ((rc = hip_check(e, "swiglu backward launch"))) return rc;
  return ok();
}

int snipop_qgemv(const void* x, int64_t ldx, int64_t tokens, const snip_qtensor* w, void* y, int y_type, int64_t ldy,
                 void* stream) {
  const char* who = "snipop_qgemv";
  if (!x || !y) return fail(SNIP_E_NULL, "%s: x and y must be non-NULL", who);
  int rc = validate_qtensor(w, "snipop_qgemv: w");
  if (rc) return rc;
  if (w->format == SNIP_BF16) return fail(SNIP_E_FORMAT, "%s: the weights must be quantized (got BF16)", who);
  if (tokens < 1 || tokens > SNIPOP_QGEMV_MAX_TOKENS)
    return fail(SNIP_E_SHAPE, "%s: %lld tokens outside 1 .. %d", who, (long long)tokens, SNIPOP_QGEMV_MAX_TOKENS);
  if (w->k % 32) return fail(SNIP_E_SHAPE, "%s: K=%lld not a multiple of 32", who, (long long)w->k);
  constexpr int64_t kMaxK = (int64_t)1 << 25;           // 16 rows of codes or tokens within 32-bit offsets
  if (w->rows > (int64_t)1 << 31 || w->k > kMaxK || ldx > kMaxK)
    return fail(SNIP_E_SHAPE, "%s: N=%lld above 2^31, or K=%lld or ldx=%lld above 2^25", who, (long long)w->rows,
                (long long)w->k, (long long)ldx);
  if (w->rows > ((int64_t)1 << 40) / w->k)              // a workgroup for 8 rows of a long K: 2^32 threads a grid
    return fail(SNIP_E_SHAPE, "%s: N=%lld times K=%lld above 2^40", who, (long long)w->rows, (long long)w->k);
  if ((rc = check_type(who, "y", y_type))) return rc;
  if (ldx < w->k || ldx % 8)
    return fail(SNIP_E_SHAPE, "%s: ldx=%lld must be >= K=%lld and a multiple of 8", who, (long long)ldx,
                (long long)w->k);
  if (ldy < w->rows || ldy > kMaxDim) return fail(SNIP_E_SHAPE, "%s: ldy=%lld must be >= N=%lld", who, (long long)ldy,
                                                 (long long)w->rows);
  if (!aligned(x, 16) || !aligned(y, 16)) return fail(SNIP_E_ALIGN, "%s: x and y must be 16-byte aligned", who);
  Gemv a;
  std::memset(&a, 0, sizeof(a));
  a.x = static_cast<const uint16_t*>(x);
  a.codes = static_cast<const uint8_t*>(w->codes);
  a.scales = static_cast<const uint8_t*>(w->scales);
  a.texp = has_texp(w->format) ? w->tensor_exp : nullptr;
  a.y = y;
  a.ldx = ldx;
  a.ldy = ldy;
  a.N = w->rows;
  a.K = w->k;
  a.M = (int32_t)tokens;
  a.y_type = y_type;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const double work = 2.0 * (double)tokens * (double)w->rows * (double)w->k;
  const int slot = timing_begin(LaunchTag{SNIPOP_LAUNCH_GEMV, w->format, -1, -1, work}, s);
  const hipError_t e = launch_gemv(w->format, a, s);
  timing_end(slot, s);
  if ((rc = hip_check(e, "gemv launch"))) return rc;
  return ok();
}

}  // extern "C"
