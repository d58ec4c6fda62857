/*
 * mhc_cross_entropy.h - C ABI of the MI355X (gfx950) softmax cross entropy of a
 * large vocabulary's logits, which are not kept, and its gradients.
 *
 *     z      = x W^T                       x [M, K] (the last norm's rows), W [V, K]; z [M, V] is not stored
 *     lse[m] = log sum over v of exp(z[m,v])                                    (fp32 [M])
 *     l[m]   = lse[m] - z[m, targets[m]],  0 where targets[m] is ignore_index   (targets int64 [M])
 *     loss   = l                           MHC_REDUCTION_NONE                   (fp32 [M])
 *            = sum of l                    MHC_REDUCTION_SUM                    (fp32 [1])
 *            = sum of l / C                MHC_REDUCTION_MEAN                   (fp32 [1])
 * with C the number of rows whose target is not ignore_index (the mean over none
 * is NaN). x and W are MHC_LINEAR_BF16 or MHC_LINEAR_F16. Sums, exponentials
 * and logarithms are fp32; an infinite logit follows the formulas (lse is +inf where one
 * is +inf and -inf where all are -inf, and G is NaN where z and lse are the same infinity).
 *
 * Gradients, from grad_loss (fp32, [M] or [1] as loss is; NULL stands for 1):
 *     s[m]        = grad_loss[m] (NONE), grad_loss (SUM), grad_loss / C (MEAN); 0 where the target is ignored
 *     G[m,v]      = rnd(s[m] (exp(z[m,v] - lse[m]) - [v = targets[m]]))
 *     grad_x      = G W                    [M, K]
 *     grad_weight = G^T x                  [V, K]
 * in the type of x; each output may be NULL (not wanted). A row with s = 0 has
 * G = 0, whatever its logits are (in grad_weight these zeros still meet its row of
 * x: an infinity or a NaN there makes NaN). G is rounded to the 16 bits that the next
 * products read: of a sum or a mean without the factor |grad_loss| or |grad_loss| / C
 * that all rows share, but for its power of two (unless grad_lse passes 2^10 of it), in fp16
 * after scaling by another power of two; the products' sums take both back, so that
 * neither a mean over many rows nor a small probability underflows.
 *
 * A target outside [0, V) that is not ignore_index makes its row's loss and
 * gradients NaN (and with them a sum, a mean and grad_weight); nothing outside W
 * is read for it.
 *
 * mhc_cross_entropy_fwd gives loss and lse. mhc_cross_entropy_bwd gives the
 * gradients from lse and makes the logits again (where lse was rounded below one of them, z - lse
 * counts as 0: no probability passes 1); it also takes grad_lse (fp32
 * [M], may be NULL), the gradient that reaches lse from its other uses:
 * G += grad_lse[m] exp(z - lse), for ignored rows too. mhc_cross_entropy_grads gives loss, lse and
 * gradients in one call, for callers that know grad_loss beforehand, and makes
 * the logits once: of a chunk of rows at a time it keeps exp(z - the largest of
 * its 64 neighbours; of 32 or 8 in the smaller kernels), rounded to fp16, in the workspace
 * (what is below 2^-40 of that largest counts as 0).
 *
 * Workspace. Both calls with gradients hold a chunk of rows of G at a time: at most
 * MHC_CROSS_ENTROPY_CHUNK_BYTES in 16 bits (or 256 rows). Where M makes several chunks and
 * grad_weight is a sum over them, its V K fp32 values are held too, which may be more than the
 * logits in 16 bits: with V = 131072 and K = 4096 1.06 GiB at 4096 rows (one chunk),
 * 2.74 at 4097, and up to 3.1 however large M is. A weight past 2^31 bytes
 * adds a chunk's M K fp32 values of grad_x, and rows along K that are no multiple of 16
 * bytes copies of x and W where they pay. The loss alone needs 8 bytes for each row
 * and 64 columns (32, 8) of a chunk, and such copies for many rows.
 *
 * The order of a sum depends on M, V, K, the type and the launch shape, on
 * nothing else: a call repeated gives the same bytes.
 *
 * Rules: as in mhc_linear.h - device pointers, contiguous row-major tensors at
 * any element alignment (slower where x or W does not start at a multiple of 16),
 * nothing allocated, calls only enqueue on `stream`. M == 0 is a successful
 * call: a sum is +0.0, a mean NaN, grad_weight +0.0. M < 0 or over 2^31 - 1, V < 1 or over
 * MHC_CROSS_ENTROPY_MAX_V, K < 1 or over MHC_LINEAR_MAX_K, another dtype, an unknown
 * reduction, a launch of MHC_LINEAR_NARROW (in the backward of MHC_LINEAR_ROWS too) or with
 * more than one part, a NULL or
 * misaligned pointer, a workspace that is too small or a size past 64 bits give
 * MHC_ERROR_INVALID_VALUE; any overlap of an output (the workspace is one) with
 * an input or another output MHC_ERROR_ALIASING; with either nothing is
 * launched. A failed launch gives MHC_ERROR_HIP. Calls that share a workspace
 * (its contents mean nothing before and after a call; aligned to 16 bytes) must
 * not overlap in time, and neither must two captured graphs of such calls.
 * launch names the kernel that makes the logits (NULL: the policy's).
 * start_event / stop_event (hipEvent_t cast to void*, each may be NULL) take the
 * start of the call's first kernel and the end of its last.
 */
#ifndef MHC_CROSS_ENTROPY_H
#define MHC_CROSS_ENTROPY_H

#include <stdint.h>

#include "mhc_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MHC_CROSS_ENTROPY_ABI_VERSION 1

#define MHC_REDUCTION_NONE 0
#define MHC_REDUCTION_SUM 1
#define MHC_REDUCTION_MEAN 2

/* Largest vocabulary accepted. */
#define MHC_CROSS_ENTROPY_MAX_V (1LL << 21)
/* Bytes of a chunk's 16-bit values. */
#define MHC_CROSS_ENTROPY_CHUNK_BYTES (1LL << 30)

int mhc_cross_entropy_abi_version(void);

/* Text of the last failure on the calling thread ("" if none). */
const char* mhc_cross_entropy_last_error_message(void);

/* Bytes of device memory a call needs as its workspace, or -1 for sizes, a
 * type or a launch that the call refuses. */
int64_t mhc_cross_entropy_fwd_workspace_bytes(int64_t M, int64_t V, int64_t K, int32_t dtype,
                                              const mhc_linear_launch* launch);
int64_t mhc_cross_entropy_bwd_workspace_bytes(int64_t M, int64_t V, int64_t K, int32_t dtype,
                                              const mhc_linear_launch* launch);
int64_t mhc_cross_entropy_grads_workspace_bytes(int64_t M, int64_t V, int64_t K, int32_t dtype,
                                                const mhc_linear_launch* launch);

mhc_status mhc_cross_entropy_fwd(const void* x, const void* weight, const int64_t* targets,
                                 float* loss, float* lse, void* workspace,
                                 int64_t workspace_bytes, int64_t M, int64_t V, int64_t K,
                                 int32_t dtype, int32_t reduction, int64_t ignore_index,
                                 void* stream, const mhc_linear_launch* launch,
                                 void* start_event, void* stop_event);

mhc_status mhc_cross_entropy_bwd(const void* x, const void* weight, const int64_t* targets,
                                 const float* lse, const float* grad_loss, const float* grad_lse,
                                 void* grad_x, void* grad_weight, void* workspace,
                                 int64_t workspace_bytes, int64_t M, int64_t V, int64_t K,
                                 int32_t dtype, int32_t reduction, int64_t ignore_index,
                                 void* stream, const mhc_linear_launch* launch,
                                 void* start_event, void* stop_event);

mhc_status mhc_cross_entropy_grads(const void* x, const void* weight, const int64_t* targets,
                                   const float* grad_loss, float* loss, float* lse, void* grad_x,
                                   void* grad_weight, void* workspace, int64_t workspace_bytes,
                                   int64_t M, int64_t V, int64_t K, int32_t dtype,
                                   int32_t reduction, int64_t ignore_index, void* stream,
                                   const mhc_linear_launch* launch, void* start_event,
                                   void* stop_event);

/* The argument checks of the three calls, on the host only. */
mhc_status mhc_cross_entropy_validate_fwd(const void* x, const void* weight,
                                          const int64_t* targets, const float* loss,
                                          const float* lse, const void* workspace,
                                          int64_t workspace_bytes, int64_t M, int64_t V, int64_t K,
                                          int32_t dtype, int32_t reduction,
                                          const mhc_linear_launch* launch);
mhc_status mhc_cross_entropy_validate_bwd(const void* x, const void* weight,
                                          const int64_t* targets, const float* lse,
                                          const float* grad_loss, const float* grad_lse,
                                          const void* grad_x, const void* grad_weight,
                                          const void* workspace, int64_t workspace_bytes,
                                          int64_t M, int64_t V, int64_t K, int32_t dtype,
                                          int32_t reduction, const mhc_linear_launch* launch);
mhc_status mhc_cross_entropy_validate_grads(const void* x, const void* weight,
                                            const int64_t* targets, const float* grad_loss,
                                            const float* loss, const float* lse,
                                            const void* grad_x, const void* grad_weight,
                                            const void* workspace, int64_t workspace_bytes,
                                            int64_t M, int64_t V, int64_t K, int32_t dtype,
                                            int32_t reduction, const mhc_linear_launch* launch);

#ifdef __cplusplus
}
#endif

#endif /* MHC_CROSS_ENTROPY_H */
