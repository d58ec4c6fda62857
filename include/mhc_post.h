/*
 * mhc_post.h - C ABI of the MI355X (gfx950) write-back of a sublayer's output
 * into the hyper-connection residual streams ("MHC Post" of the page "Add
 * batch-invariant h_aggregate kernel", RL-Kernel pull request 366, which names
 * the step and defines nothing of it), and its backward.
 *
 *     residual [T, n, H] bf16    the streams, n in {2, 4, 8}
 *     comb     [T, n, n] fp32    mixing matrix, row-major (row i makes stream i)
 *     post     [T, n]    fp32    write-back gates
 *     y        [T, H]    bf16    the sublayer's output
 *     out      [T, n, H] bf16
 *     out[t,i,h] = sum_j comb[t,i,j] * residual[t,j,h] + post[t,i] * y[t,h]
 *
 * Backward, from grad_out [T, n, H] bf16:
 *     grad_residual[t,j,h] = sum_i comb[t,i,j] * grad_out[t,i,h]        bf16
 *     grad_y[t,h]          = sum_i post[t,i] * grad_out[t,i,h]          bf16
 *     grad_comb[t,i,j]     = sum_h grad_out[t,i,h] * residual[t,j,h]    fp32
 *     grad_post[t,i]       = sum_h grad_out[t,i,h] * y[t,h]             fp32
 *
 * Every sum is held in fp32 (one fused multiply-add a term, in ascending
 * order of the summed stream) and each bf16 result is rounded once, to
 * nearest even. The sums over h follow one order that depends only on H, so
 * a token's results never depend on T or on the other tokens.
 *
 * Rules: as in mhc_h_aggregate.h - device pointers, contiguous row-major
 * tensors, any element alignment, nothing allocated, calls only enqueue on
 * `stream`; T == 0 is a successful no-op; n not in {2, 4, 8}, T < 0, H < 1,
 * H > MHC_MAX_H, a NULL or misaligned pointer or a size past 64 bits give
 * MHC_ERROR_INVALID_VALUE, any overlap of an output with an input or another
 * output MHC_ERROR_ALIASING, with nothing launched; a failed launch gives
 * MHC_ERROR_HIP. start_event / stop_event (hipEvent_t cast to void*, each may
 * be NULL) take the kernel's own start and end.
 */
#ifndef MHC_POST_H
#define MHC_POST_H

#include <stdint.h>

#include "mhc_h_aggregate.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MHC_POST_ABI_VERSION 1

int mhc_post_abi_version(void);

/* Text of the last failure on the calling thread ("" if none). */
const char* mhc_post_last_error_message(void);

mhc_status mhc_post_fwd(const uint16_t* residual, const float* comb, const float* post,
                        const uint16_t* y, uint16_t* out, int64_t T, int32_t n, int64_t H,
                        void* stream, void* start_event, void* stop_event);

mhc_status mhc_post_bwd(const uint16_t* grad_out, const uint16_t* residual, const float* comb,
                        const float* post, const uint16_t* y, uint16_t* grad_residual,
                        float* grad_comb, float* grad_post, uint16_t* grad_y, int64_t T,
                        int32_t n, int64_t H, void* stream, void* start_event,
                        void* stop_event);

/* The argument checks of the two calls, on the host only. */
mhc_status mhc_post_validate_fwd(const uint16_t* residual, const float* comb, const float* post,
                                 const uint16_t* y, const uint16_t* out, int64_t T, int32_t n,
                                 int64_t H);
mhc_status mhc_post_validate_bwd(const uint16_t* grad_out, const uint16_t* residual,
                                 const float* comb, const float* post, const uint16_t* y,
                                 const uint16_t* grad_residual, const float* grad_comb,
                                 const float* grad_post, const uint16_t* grad_y, int64_t T,
                                 int32_t n, int64_t H);

#ifdef __cplusplus
}
#endif

#endif /* MHC_POST_H */
