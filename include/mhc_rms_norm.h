/*
 * mhc_rms_norm.h - C ABI of the MI355X (gfx950) root-mean-square norm in front
 * of a hyper-connected sublayer, with the residual's addition or the streams'
 * collapse in the same pass and an optional 8-bit output with scales; and its
 * backward.
 *
 * Forward. One row t of H elements comes from one of three sources:
 *     x        [T, H]                        s = x
 *     x + r    [T, H] twice                  s = rnd(x + r)
 *     streams  [T, n, H] with pre [T, n]     s = rnd(the collapse of mhc_h_aggregate.h, its bits)
 * where rnd rounds the fp32 value to the storage type (nearest even). Then
 *     rstd[t]  = 1 / sqrt(mean over h of s[t,h]^2 + eps)
 *     v[t,h]   = s[t,h] * rstd[t] * weight[h]
 * and the output is, by out_format,
 *     MHC_NORM_SAME      out[t,h] = rnd(v[t,h])
 *     MHC_NORM_E4M3_ROW  scales[t] = max(amax / 448, 2^-126), amax over the row of |v|   (fp32 [T])
 *                        out[t,h] = e4m3(v[t,h] * (1 / scales[t]))
 *     MHC_NORM_E4M3_MX   for each block of 32 consecutive columns (the last may be
 *                        short) p = the smallest integer in [-127, 127] with
 *                        amax over the block of |v| <= 448 * 2^p;
 *                        scales[t][h / 32] = p + 127, the e8m0 byte of 2^p
 *                        ([T, ceil(H / 32)] bytes; 255, a NaN, where amax is infinite);
 *                        out[t,h] = e4m3(v[t,h] * 2^-p)
 * e4m3 is the OCP format (4 exponent and 3 mantissa bits, largest 448), rounded
 * to nearest even; by the choice of scale nothing saturates. A NaN stays a NaN.
 * s and rstd are written where `stored` and `rstd` are given (stored only where
 * s is new, i.e. with a residual or pre).
 *
 * Backward of the MHC_NORM_SAME output, from grad_y [T, H], s, rstd and, where
 * given, grad_stored [T, H] (the gradient that reaches s from its other uses):
 *     u       = grad_y * weight
 *     grad_x  = rnd(rstd * (u - s * (mean over h of u * s) * rstd^2) + grad_stored)
 *     grad_weight[h] = sum over t of grad_y * s * rstd                   (fp32 [H])
 * grad_x is the gradient of x and of r alike, or of the collapsed row, which
 * mhc_h_aggregate_bwd takes further.
 *
 * Values are fp32 in registers and sums are held in fp32: a row whose sum of
 * squares passes the range of fp32 (values from about 1.8e19 / sqrt(H) on) has
 * rstd 0, and squares below 2^-149 count as 0 (with eps 0 a row of nothing else
 * has rstd inf). The sums over h
 * follow an order that depends only on H, so a row's bytes never depend on T or
 * on other rows; grad_weight sums rows in an order that depends only on T and H.
 *
 * Types: dtype (of x, r, s, grad_y, grad_stored, grad_x and the MHC_NORM_SAME
 * output) is MHC_NORM_F32, MHC_NORM_BF16 or MHC_NORM_F16; streams are bf16.
 * weight_dtype is dtype or MHC_NORM_F32. 16-bit tensors are raw bit patterns.
 *
 * Rules: as in mhc_h_aggregate.h - device pointers, contiguous row-major tensors
 * at any element alignment, nothing allocated, calls only enqueue on `stream`.
 * T == 0 is a successful call (the backward then writes grad_weight = +0.0).
 * T < 0, H < 1, H > MHC_MAX_H, an unknown type, eps negative or not finite,
 * residual and pre together, pre with n not in {2, 4, 8} or dtype not bf16, n
 * not 0 without pre, stored without residual or pre, scales missing or given
 * where the format has none, a NULL or misaligned pointer, a workspace that is
 * too small or a size past 64 bits give MHC_ERROR_INVALID_VALUE; any overlap
 * of an output (the workspace is one) with an input or another output
 * MHC_ERROR_ALIASING; with either nothing is launched. A failed launch gives
 * MHC_ERROR_HIP. start_event / stop_event (hipEvent_t cast to void*, each may be
 * NULL) take the start of the call's first kernel and the end of its last.
 */
#ifndef MHC_RMS_NORM_H
#define MHC_RMS_NORM_H

#include <stdint.h>

#include "mhc_h_aggregate.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MHC_NORM_ABI_VERSION 1

/* Storage types. */
#define MHC_NORM_F32 0
#define MHC_NORM_BF16 1
#define MHC_NORM_F16 2

/* Output formats. */
#define MHC_NORM_SAME 0
#define MHC_NORM_E4M3_ROW 1
#define MHC_NORM_E4M3_MX 2

int mhc_rms_norm_abi_version(void);

/* Text of the last failure on the calling thread ("" if none). */
const char* mhc_rms_norm_last_error_message(void);

/* residual, pre, stored, rstd and scales may be NULL as described above. */
mhc_status mhc_rms_norm_fwd(const void* x, const void* residual, const float* pre, int32_t n,
                            const void* weight, int32_t weight_dtype, float eps, void* out,
                            void* scales, void* stored, float* rstd, int64_t T, int64_t H,
                            int32_t dtype, int32_t out_format, void* stream, void* start_event,
                            void* stop_event);

/* Bytes of device memory the backward needs as its workspace (contents before
 * and after a call mean nothing; calls that share one must not overlap in
 * time, and neither must two captured graphs of such calls), or -1 for a T or H
 * that is out of range. */
int64_t mhc_rms_norm_bwd_workspace_bytes(int64_t T, int64_t H);

mhc_status mhc_rms_norm_bwd(const void* grad_y, const void* stored, const void* weight,
                            int32_t weight_dtype, const float* rstd, const void* grad_stored,
                            void* grad_x, float* grad_weight, void* workspace,
                            int64_t workspace_bytes, int64_t T, int64_t H, int32_t dtype,
                            void* stream, void* start_event, void* stop_event);

/* The argument checks of the two calls, on the host only. */
mhc_status mhc_rms_norm_validate_fwd(const void* x, const void* residual, const float* pre,
                                     int32_t n, const void* weight, int32_t weight_dtype,
                                     float eps, const void* out, const void* scales,
                                     const void* stored, const float* rstd, int64_t T, int64_t H,
                                     int32_t dtype, int32_t out_format);
mhc_status mhc_rms_norm_validate_bwd(const void* grad_y, const void* stored, const void* weight,
                                     int32_t weight_dtype, const float* rstd,
                                     const void* grad_stored, const void* grad_x,
                                     const float* grad_weight, const void* workspace,
                                     int64_t workspace_bytes, int64_t T, int64_t H,
                                     int32_t dtype);

#ifdef __cplusplus
}
#endif

#endif /* MHC_RMS_NORM_H */
