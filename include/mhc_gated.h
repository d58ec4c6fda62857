/*
 * mhc_gated.h - C ABI of the MI355X (gfx950) gated feed-forward block of a
 * hyper-connected sublayer: both projections, the activation and the product of
 * the two in one kernel, and its backward. The block's last projection is
 * mhc_linear_fwd.
 *
 *     gate = x Wg^T + gate_bias          x [M, K], Wg and Wu [N, K], biases [N]
 *     up   = x Wu^T + up_bias
 *     out  = act(gate) * up              out, gate, up [M, N]
 * with dtype, the scales and act as in mhc_linear.h (the scales of both weights
 * are of the same kind). Sums over k and the epilogue are fp32 (of 8-bit integers
 * exact); out, gate and up are each rounded once, and out is made of the values
 * before that rounding. The biases, and gate and up as outputs, may be NULL.
 *
 * Backward (16-bit types), from grad_out [M, N] and the forward's gate and up (as
 * the forward wrote them, in 16 bits):
 *     dg = rnd((grad_out * up) * act'(gate))   (rounded: the next products read 16 bits)
 *     du = rnd(grad_out * act(gate))
 *     grad_x = dg Wg + du Wu                   (one sum, rounded once)       [M, K]
 *     grad_gate_weight = dg^T x,  grad_up_weight = du^T x                    [N, K]
 *     grad_gate_bias, grad_up_bias = the sums over m of dg and du unrounded  [N]
 * in the type of x; each output may be NULL (not wanted; the weights' gradients
 * only together). act' of an infinite gate is its limit, 0 or 1; the products
 * with it follow fp32's rules (infinity times 0 is NaN).
 *
 * Where dg and du together pass 2^31 - 1 bytes (4 M times N rounded up to 64: 32768 rows x 16384)
 * the weights' gradients take about two thirds longer: 32768 x 4096 with 16320
 * columns 7.4 ms, with 16384 12.4.
 *
 * The order of a sum depends on M, N, K, the type and the launch shape, on
 * nothing else: a call repeated gives the same bytes. With a launch that names
 * a tile kernel and splits = 1 a row's bytes do not depend on M either.
 *
 * Rules: as in mhc_linear.h - device pointers, contiguous row-major tensors at
 * any element alignment (slower where x or a weight does not start at a multiple of
 * 16), nothing allocated, calls only enqueue on `stream`. M == 0 is a successful
 * call (the backward then writes the weights' and biases' gradients = +0.0). N over 2^30 - 1,
 * in the backward over MHC_GATED_MAX_BWD_N, a launch of MHC_LINEAR_NARROW, one
 * weight's gradient without the other's, and what mhc_linear.h names of sizes, types,
 * pointers, scales, launches and workspaces give MHC_ERROR_INVALID_VALUE; any
 * overlap of an output (the workspace is one) with an input or another output
 * MHC_ERROR_ALIASING; with either nothing is launched. A failed launch gives
 * MHC_ERROR_HIP. Calls that share a workspace (its contents mean nothing before
 * and after a call) must not overlap in time, and neither must two captured
 * graphs of such calls. start_event / stop_event (hipEvent_t cast to void*, each
 * may be NULL) take the start of the call's first kernel and the end of its last.
 */
#ifndef MHC_GATED_H
#define MHC_GATED_H

#include <stdint.h>

#include "mhc_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MHC_GATED_ABI_VERSION 1

/* Largest N of the backward, whose sum for grad_x runs over both blocks of N. */
#define MHC_GATED_MAX_BWD_N (1LL << 20)

int mhc_gated_abi_version(void);

/* Text of the last failure on the calling thread ("" if none). */
const char* mhc_gated_last_error_message(void);

/* The launch a forward call with these sizes would use, every field filled in;
 * host only. launch may be NULL; its kernels' tiles are half as many columns of
 * out wide as mhc_linear.h names. */
mhc_status mhc_gated_plan(int64_t M, int64_t N, int64_t K, int32_t dtype,
                          const mhc_linear_launch* launch, mhc_linear_launch* plan);

/* Bytes of device memory a call needs as its workspace, or -1 for sizes, a
 * type or a launch that the call refuses. */
int64_t mhc_gated_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t dtype,
                                      const mhc_linear_launch* launch);
int64_t mhc_gated_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t dtype);

mhc_status mhc_gated_fwd(const void* x, const void* x_scales, const void* gate_weight,
                         const void* gate_scales, const void* up_weight, const void* up_scales,
                         const void* gate_bias, const void* up_bias, void* out, void* gate,
                         void* up, void* workspace, int64_t workspace_bytes, int64_t M, int64_t N,
                         int64_t K, int32_t dtype, int32_t act, void* stream,
                         const mhc_linear_launch* launch, void* start_event, void* stop_event);

mhc_status mhc_gated_bwd(const void* grad_out, const void* x, const void* gate_weight,
                         const void* up_weight, const void* gate, const void* up, void* grad_x,
                         void* grad_gate_weight, void* grad_up_weight, void* grad_gate_bias,
                         void* grad_up_bias, void* workspace, int64_t workspace_bytes, int64_t M,
                         int64_t N, int64_t K, int32_t dtype, int32_t act, void* stream,
                         void* start_event, void* stop_event);

/* The argument checks of the two calls, on the host only. */
mhc_status mhc_gated_validate_fwd(const void* x, const void* x_scales, const void* gate_weight,
                                  const void* gate_scales, const void* up_weight,
                                  const void* up_scales, const void* gate_bias,
                                  const void* up_bias, const void* out, const void* gate,
                                  const void* up, const void* workspace, int64_t workspace_bytes,
                                  int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t act,
                                  const mhc_linear_launch* launch);
mhc_status mhc_gated_validate_bwd(const void* grad_out, const void* x, const void* gate_weight,
                                  const void* up_weight, const void* gate, const void* up,
                                  const void* grad_x, const void* grad_gate_weight,
                                  const void* grad_up_weight, const void* grad_gate_bias,
                                  const void* grad_up_bias, const void* workspace,
                                  int64_t workspace_bytes, int64_t M, int64_t N, int64_t K,
                                  int32_t dtype, int32_t act);

#ifdef __cplusplus
}
#endif

#endif /* MHC_GATED_H */
