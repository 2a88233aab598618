/*
 * snip_ops.h -- the operators around the quantized linear layers of a
 * Llama-like block, in the same library as snip.h (libsnip): RMS norm with
 * the residual's addition, SwiGLU, both with an output quantized in the
 * launch and a backward pass, and the product of one to sixteen tokens with
 * block-scaled weights.
 *
 * Conventions are those of snip.h (caller-owned buffers, validation before
 * any HIP call, int status, snip_last_error(), work enqueued on `stream`),
 * and its descriptors, formats and status codes are used. What differs:
 *   Types       A matrix argument is a device pointer with an element type
 *               (SNIPOP_BF16 / SNIPOP_F32) and a leading dimension in
 *               elements: ld >= cols, ld % 8 == 0 for bf16, ld % 4 == 0 for
 *               fp32; the pointer is 16-byte aligned. `cols` itself need not
 *               be a multiple of anything unless an output is quantized.
 *   Arithmetic  fp32 throughout (sums, statistics, exponentials); a value is
 *               rounded once, to nearest even, when it is stored as bf16. A
 *               row whose sum of squares leaves fp32 (values of 1e17 and
 *               more) has r = 0. sigmoid is within 7 * 2^-24 of its value, and
 *               0 where exp(-gate) leaves fp32 (gate below -88).
 *   Overlap     An output may be the very matrix that an input is (same
 *               pointer, type and leading dimension) where the entry says
 *               so; any other overlap is undefined.
 */
#ifndef SNIP_OPS_H
#define SNIP_OPS_H

#include "snip.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of matrix arguments */
#define SNIPOP_BF16  0
#define SNIPOP_F32   1

/* Largest row of the norm (a row is held in registers). */
#define SNIPOP_NORM_MAX_COLS   16384
/* Most tokens of one snipop_qgemv call. */
#define SNIPOP_QGEMV_MAX_TOKENS   16

/* launch kinds in the timing records (snip_timing_*), next to SNIP_LAUNCH_* */
#define SNIPOP_LAUNCH_NORM   5  /* norm forward / backward; work: elements        */
#define SNIPOP_LAUNCH_GATE   6  /* SwiGLU forward / backward; work: elements      */
#define SNIPOP_LAUNCH_GEMV   7  /* tokens x weights product; work: 2*M*N*K flop   */

/* RMS norm of a residual stream:
 *   h = x + res;  r = 1 / sqrt(mean_c(h^2) + eps);  y = h * r * gamma
 * per row of [rows][cols], with y stored, quantized, or both.
 *   x          device, x_type, ldx.
 *   res        device, res_type, ldr; NULL: h = x.
 *   gamma      device [cols], gamma_type, 16-byte aligned.
 *   eps        >= 0, finite.
 *   h          device, h_type, ldh, or NULL (not stored). May be x or res
 *              itself: the residual stream updated in place. The backward
 *              pass reads this h, so a training step keeps it as it is until
 *              then: no later norm may update that buffer in place.
 *   y          device, y_type, ldy, or NULL.
 *   rstd       device fp32 [rows] (r, for the backward pass) or NULL.
 *   out        host descriptor or NULL: y quantized row-wise in out->format
 *              (NVFP4, FP8_E4M3 or MXFP4; rows, k = cols; cols % 16 == 0,
 *              MXFP4 % 32), as snip_quantize would quantize a tensor holding
 *              the fp32 y: a GEMM operand without another read of y.
 *   rounding, seed, tensor_id, amax_in, stats  as snip_quantize, for `out`.
 *              amax_in NULL (NVFP4, FP8): max|y| comes from an extra pass
 *              that reads x, res and gamma.
 *   ws         device, snipop_rmsnorm_fwd_workspace() bytes; needed only for
 *              stats, or to find max|y|.
 *   rows > 0; 0 < cols <= SNIPOP_NORM_MAX_COLS. At least one of h, y, rstd,
 *   out must be given.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, WORKSPACE, HIP. */
int snipop_rmsnorm_fwd(const void* x, int x_type, int64_t ldx,
                       const void* res, int res_type, int64_t ldr,
                       const void* gamma, int gamma_type,
                       int64_t rows, int64_t cols, float eps,
                       void* h, int h_type, int64_t ldh, void* y, int y_type, int64_t ldy, float* rstd,
                       const snip_qtensor* out, int rounding, uint64_t seed, uint32_t tensor_id,
                       const float* amax_in, snip_stats* stats,
                       void* ws, size_t ws_bytes, void* stream);

/* Backward of the norm, with xh = h * r:
 *   dx = r * (dy * gamma - xh * mean_c(dy * gamma * xh)) + dres
 *   dgamma = sum over rows of dy * xh
 * dx is the gradient of x and of res alike. A quantized output passes its
 * gradient straight through (dy is the gradient of y).
 *   dy         device, dy_type, lddy.
 *   h          device, h_type, ldh: the forward's h (x where there was no res).
 *   rstd       device fp32 [rows] from the forward.
 *   dres       device, dres_type, lddres, or NULL: the gradient that reaches h
 *              along the residual stream.
 *   dx         device, dx_type, lddx, or NULL. May be dy or dres itself.
 *   dgamma     device fp32 [cols], overwritten, or NULL. Summed in a fixed
 *              order: the same inputs give the same bits.
 *   ws         device, snipop_rmsnorm_bwd_workspace() bytes (with dgamma).
 *   At least one of dx and dgamma must be given; shapes as the forward's.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, WORKSPACE, HIP. */
int snipop_rmsnorm_bwd(const void* dy, int dy_type, int64_t lddy, const void* h, int h_type, int64_t ldh,
                       const void* gamma, int gamma_type, const float* rstd,
                       const void* dres, int dres_type, int64_t lddres, int64_t rows, int64_t cols,
                       void* dx, int dx_type, int64_t lddx, float* dgamma,
                       void* ws, size_t ws_bytes, void* stream);

/* SwiGLU: y = gate * sigmoid(gate) * up, elementwise on [rows][cols], stored,
 * quantized, or both.
 *   gate, up   device, one type, own leading dimensions (the two halves of
 *              one product's output, for instance).
 *   y, out, rounding, seed, tensor_id, amax_in, stats, ws  as
 *              snipop_rmsnorm_fwd. y may be gate or up itself, also where the
 *              maximum is computed (the pass for it writes nothing).
 *   rows > 0, 0 < cols <= 2^31. One of y and out must be given.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, WORKSPACE, HIP. */
int snipop_swiglu_fwd(const void* gate, int64_t ldg, const void* up, int64_t ldu, int type,
                      int64_t rows, int64_t cols, void* y, int y_type, int64_t ldy,
                      const snip_qtensor* out, int rounding, uint64_t seed, uint32_t tensor_id,
                      const float* amax_in, snip_stats* stats,
                      void* ws, size_t ws_bytes, void* stream);

/* Backward of SwiGLU, with s = sigmoid(gate):
 *   dgate = dy * up * s * (1 + gate * (1 - s));  dup = dy * gate * s
 *   dy         device, dy_type, lddy; gate, up as the forward's.
 *   dgate, dup device, d_type, own leading dimensions, or NULL (not both).
 *              Each may be dy, gate or up itself.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, HIP. */
int snipop_swiglu_bwd(const void* dy, int dy_type, int64_t lddy, const void* gate, int64_t ldg,
                      const void* up, int64_t ldu, int type, int64_t rows, int64_t cols,
                      void* dgate, int64_t lddg, void* dup, int64_t lddu, int d_type, void* stream);

/* y[tokens][N] = x[tokens][K] . dequant(w)[N][K]^T for a few tokens: a decode
 * step's linear layer, with the activations left in bf16.
 *   x          device bf16, ldx; 1 <= tokens <= SNIPOP_QGEMV_MAX_TOKENS.
 *   w          host descriptor: N = w->rows, K = w->k; any format but BF16
 *              (FP8_E4M3, NVFP4, MXFP4 and the FP4 variants); K % 32 == 0;
 *              N <= 2^31, K and ldx <= 2^25, N K <= 2^40.
 *   y          device, y_type, ldy >= N.
 * Products are exact, over the whole range of a scale, and sums are fp32, in a
 * fixed order that depends on the shapes, and for E8M0 and bf16 scales on
 * whether some of 16 to 64 neighbouring rows lie at the ends of their range
 * (E8M0 from 2^126, bf16 from 2^125 and below 2^-125). A block is summed before
 * its scale, and a row before 2^tensor_exp: |x| below 2^90 keeps these sums
 * within fp32 at any length. No workspace.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, HIP. */
int snipop_qgemv(const void* x, int64_t ldx, int64_t tokens, const snip_qtensor* w,
                 void* y, int y_type, int64_t ldy, void* stream);

/* Workspace bytes of the calls above (0 on invalid arguments). format: that
 * of `out`. */
size_t snipop_rmsnorm_fwd_workspace(int64_t rows, int64_t cols, int format);
size_t snipop_rmsnorm_bwd_workspace(int64_t rows, int64_t cols);
size_t snipop_swiglu_fwd_workspace(int64_t rows, int64_t cols, int format);

#ifdef __cplusplus
}
#endif

#endif /* SNIP_OPS_H */
