/*
 * mhc_linear.h - C ABI of the MI355X (gfx950) matrix product of a
 * hyper-connected sublayer, with bias, activation and residual in its
 * epilogue, and its backward.
 *
 *     z   = x W^T + bias               x [M, K], W [N, K], bias [N]
 *     out = act(z) + residual          residual, out, z [M, N]
 *     act: MHC_ACT_NONE v, _RELU max(v, 0), _SILU v / (1 + exp(-v)),
 *          _GELU v * (1 + erf(v / sqrt 2)) / 2
 *          (at v = -inf RELU and GELU give their limit 0, SILU its formula's NaN)
 *
 * dtype says what x and W are:
 *     MHC_LINEAR_BF16, MHC_LINEAR_F16   16-bit values; bias, residual, out and z in the same type
 *     MHC_LINEAR_E4M3_ROW               e4m3 codes with fp32 scales x_scales [M], weight_scales [N]
 *     MHC_LINEAR_E4M3_MX                e4m3 codes with e8m0 scales x_scales [M, ceil(K/32)],
 *                                       weight_scales [N, ceil(K/32)], one for 32 consecutive k
 *     MHC_LINEAR_I8_ROW                 8-bit integers with fp32 scales x_scales [M], weight_scales [N]
 * and the 8-bit forms (the outputs of mhc_rms_norm_fwd) take and give bf16
 * otherwise. Sums over k and the epilogue are fp32, and out and z are each
 * rounded once. 16-bit products enter the sum exactly; the sum of 8-bit integers
 * is an exact 32-bit integer, rounded to fp32 once; of e4m3 products the
 * matrix instruction drops, in each group of 8 consecutive k, the bits below
 * 2^-13 of the largest product's power of two (so a group is off by at most
 * 7 * 2^-13 of its largest product). bias, residual and z may be NULL (absent).
 *
 * Backward (16-bit types), from grad_out [M, N] and the forward's z (needed
 * unless act is MHC_ACT_NONE; as the forward wrote it, in 16 bits):
 *     gz          = rnd(grad_out * act'(z))      (rounded: the next products read 16 bits)
 *     grad_x      = gz W                         [M, K]
 *     grad_weight = gz^T x                       [N, K]
 *     grad_bias   = sum over m of grad_out * act'(z), unrounded, in fp32     [N]
 * in the type of x; each output may be NULL (not wanted). The residual's
 * gradient is grad_out itself. act' of an infinite z is its limit, 0 or 1 (in
 * fp16 a z past +-65520 is stored as an infinity).
 *
 * The order of a sum over k depends on M, N, K, the type and the launch shape,
 * on nothing else: a call repeated gives the same bytes. With a launch that
 * names a tile kernel and splits = 1, a row's bytes do not depend on M either;
 * with the policy's launch they do (from 16 to 17 rows, for one), and the
 * backward always takes the policy's. With 8-bit integers no launch and no M
 * changes a row's bytes.
 *
 * Rules: as in mhc_h_aggregate.h - device pointers, contiguous row-major
 * tensors at any element alignment (the same bytes, in two to three times
 * the time where x or W does not start at a multiple of 16), nothing allocated,
 * calls only enqueue on `stream`. M == 0 is a successful call (the backward then writes grad_weight
 * and grad_bias = +0.0). M < 0, N < 1, K < 1, K > MHC_LINEAR_MAX_K (with 8-bit
 * integers over MHC_LINEAR_MAX_K_I8), M or N
 * over 2^31 - 1 (in the backward, which sums over them, over
 * MHC_LINEAR_MAX_K), N over 2^26 with M <= 16, more than 2^23 tiles (of 256 x
 * 256: 2^21) in one launch, an unknown dtype or act, scales missing or given
 * where the type has none, a NULL or misaligned pointer, a launch that does not
 * exist, a workspace that is too small or a size past 64 bits give
 * MHC_ERROR_INVALID_VALUE; any overlap of an output (the workspace is one) with
 * an input or another output MHC_ERROR_ALIASING; with either nothing is
 * launched. A failed launch gives MHC_ERROR_HIP. The workspace is aligned to 16
 * bytes (the sums of a split call are in it, and copies of long operands whose
 * rows are not whole pieces of 16 bytes; the backward's is sized for any act
 * and all three gradients, with M x N values of gz in it); its contents mean nothing before and
 * after a call; calls that share one must not overlap in time, and neither must
 * two captured graphs of such calls. start_event / stop_event (hipEvent_t cast
 * to void*, each may be NULL) take the start of the call's first kernel and the
 * end of its last.
 */
#ifndef MHC_LINEAR_H
#define MHC_LINEAR_H

#include <stdint.h>

#include "mhc_h_aggregate.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MHC_LINEAR_ABI_VERSION 1

#define MHC_LINEAR_BF16 1
#define MHC_LINEAR_F16 2
#define MHC_LINEAR_E4M3_ROW 3
#define MHC_LINEAR_E4M3_MX 4
#define MHC_LINEAR_I8_ROW 6 /* 5 is no type */

#define MHC_ACT_NONE 0
#define MHC_ACT_RELU 1
#define MHC_ACT_SILU 2
#define MHC_ACT_GELU 3

/* Longest sum accepted. */
#define MHC_LINEAR_MAX_K (1LL << 21)
/* And of 8-bit integers, whose sums are held in 32 bits: 131071 (-128)^2 < 2^31. */
#define MHC_LINEAR_MAX_K_I8 131071

/* Kernels of the forward (mhc_linear_launch.kernel). */
#define MHC_LINEAR_ROWS 1    /* up to 16 rows of x: the weight is streamed once */
#define MHC_LINEAR_NARROW 2  /* tiles of 64 x 32 */
#define MHC_LINEAR_SMALL 3   /* tiles of 64 x 64 */
#define MHC_LINEAR_MEDIUM 4  /* tiles of 128 x 128 */
#define MHC_LINEAR_LARGE 5   /* tiles of 256 x 256 */
#define MHC_LINEAR_SHORT 7   /* tiles of 32 x 64; 6 is no kernel */

/* Launch shape: kernel and the number of parts that the sum over k is split
 * into (tile kernels: 1..64; parts are joined in ascending order by a second
 * kernel). A field of 0 lets the policy choose. */
typedef struct mhc_linear_launch {
  int32_t kernel;
  int32_t splits;
} mhc_linear_launch;

int mhc_linear_abi_version(void);

/* Text of the last failure on the calling thread ("" if none). */
const char* mhc_linear_last_error_message(void);

/* The launch a forward call with these sizes would use, every field filled in;
 * host only. launch may be NULL. */
mhc_status mhc_linear_plan(int64_t M, int64_t N, int64_t K, int32_t dtype,
                           const mhc_linear_launch* launch, mhc_linear_launch* plan);

/* Bytes of device memory a call needs as its workspace, or -1 for sizes, a
 * type or a launch that the call refuses. */
int64_t mhc_linear_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t dtype,
                                       const mhc_linear_launch* launch);
int64_t mhc_linear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t dtype);

mhc_status mhc_linear_fwd(const void* x, const void* x_scales, const void* weight,
                          const void* weight_scales, const void* bias, const void* residual,
                          void* out, void* z, void* workspace, int64_t workspace_bytes, int64_t M,
                          int64_t N, int64_t K, int32_t dtype, int32_t act, void* stream,
                          const mhc_linear_launch* launch, void* start_event, void* stop_event);

mhc_status mhc_linear_bwd(const void* grad_out, const void* x, const void* weight, const void* z,
                          void* grad_x, void* grad_weight, void* grad_bias, void* workspace,
                          int64_t workspace_bytes, int64_t M, int64_t N, int64_t K, int32_t dtype,
                          int32_t act, void* stream, void* start_event, void* stop_event);

/* The argument checks of the two calls, on the host only. */
mhc_status mhc_linear_validate_fwd(const void* x, const void* x_scales, const void* weight,
                                   const void* weight_scales, const void* bias,
                                   const void* residual, const void* out, const void* z,
                                   const void* workspace, int64_t workspace_bytes, int64_t M,
                                   int64_t N, int64_t K, int32_t dtype, int32_t act,
                                   const mhc_linear_launch* launch);
mhc_status mhc_linear_validate_bwd(const void* grad_out, const void* x, const void* weight,
                                   const void* z, const void* grad_x, const void* grad_weight,
                                   const void* grad_bias, const void* workspace,
                                   int64_t workspace_bytes, int64_t M, int64_t N, int64_t K,
                                   int32_t dtype, int32_t act);

#ifdef __cplusplus
}
#endif

#endif /* MHC_LINEAR_H */
