/*
 * gemm_ops.h -- C ABI of the operators beside the GEMM of gemm.h: the gated
 * feed-forward block of a language model, its backward pass, its products
 * from 4-bit weights, and the orthogonalised update of its matrices.
 *
 * Types: GEMM_F16 or GEMM_BF16 for every 16-bit tensor of a call; sums run in
 * fp32.  Matrices are row-major; ld* is the distance between rows in elements
 * (a row's elements are contiguous).
 *
 * Ownership, errors, streams: as in gemm.h.  The caller owns every buffer,
 * the workspaces included; argument checks run on the host before any launch,
 * so a rejected call writes nothing; a kernel that stops making progress
 * records GEMM_ERR_TIMEOUT, which gemm_ops_check_error reports.  Calls are
 * asynchronous on `stream` (a cudaStream_t of the handle's device; NULL =
 * legacy default stream), allocate nothing and do not synchronize.  A handle
 * holds no data between calls: the operators may be called with it on any
 * number of streams and from any number of host threads, as long as calls that
 * overlap on the GPU have workspaces of their own (gemm_ops_set_watchdog,
 * _check_error and _destroy: while no other thread uses the handle).
 *
 * Every pointer must be device memory of the handle's device; outputs and
 * workspaces must not overlap inputs or one another (an output may have other
 * columns of an input's matrix: rows of one pitch that share no element).
 * Lengths are at most 2^31 - 4096 (F and the N of 4-bit weights: 2^30 - 1) and
 * row distances below 2^30 (free where a function says so).  Results do not
 * depend on timing: no sum is taken in the order in which parts arrive.
 */
#ifndef GB300_GEMM_OPS_H_
#define GB300_GEMM_OPS_H_

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gemm_ops_s* gemm_ops_t;

typedef enum {
    GEMM_F16 = 0,
    GEMM_BF16 = 1,
    GEMM_F32 = 2 /* gemm_orthogonalize's input and output only */
} gemm_dtype_t;

/* The gate's activation.  GELU is its tanh form,
 * g / 2 (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))). */
typedef enum {
    GEMM_ACT_SILU = 0,
    GEMM_ACT_GELU_TANH = 1,
    GEMM_ACT_RELU = 2
} gemm_act_t;

/* Create a handle bound to CUDA device `device` (an sm_103 part): queries the
 * device, sets the kernels' attributes and allocates a 16-byte watchdog
 * record.  *out receives the handle, or NULL on error. */
GEMM_API gemm_status_t gemm_ops_create(gemm_ops_t* out, int device);
/* Release it (NULL: no-op).  Not while work launched with it is running. */
GEMM_API gemm_status_t gemm_ops_destroy(gemm_ops_t ops);

/* Synchronize, read and clear the watchdog record: GEMM_OK, GEMM_ERR_TIMEOUT
 * or GEMM_ERR_CUDA. */
GEMM_API gemm_status_t gemm_ops_check_error(gemm_ops_t ops);
/* The record last read: status, wait site, CTA, work item. */
GEMM_API gemm_status_t gemm_ops_last_error_detail(gemm_ops_t ops, uint32_t detail[4]);
/* As gemm_plan_set_watchdog: the longest single wait inside a kernel (0: the
 * default of 2 s), and the k-block whose load the first unit skips (-1: none;
 * for testing that a stuck wait ends). */
GEMM_API gemm_status_t gemm_ops_set_watchdog(gemm_ops_t ops, uint64_t timeout_ns,
                                             int32_t skip_k_block);
/* Kernels launched through the handle so far. */
GEMM_API uint64_t gemm_ops_launch_count(gemm_ops_t ops);

/* The gated feed-forward block on T tokens:
 *
 *     g = x Wg^T,  u = x Wu^T,  h = act(g) * u,  y = h Wd^T
 *
 *   x      : [T, D];   y : [T, D]
 *   w_in   : [2 F, D]: the F rows of Wg, then the F rows of Wu
 *   w_down : [D, F] (Wd)
 *   gu     : [T, 2 F] contiguous, or NULL: receives g (columns 0 .. F-1) and u
 *            for the backward pass
 * g, u and act(g) * u are fp32 until h is rounded to 16 bits as an operand of
 * the second product.  D and F are multiples of 8, pointers 16-byte aligned,
 * row distances multiples of 8 (GEMM_ERR_ALIGNMENT otherwise).  T == 0:
 * nothing to do; D == 0: gu is zero; F == 0: y is zero.  Infinities and NaN go
 * where the formula puts them (silu and gelu of a gate of -inf are NaN).
 * workspace: gemm_gated_ffn_workspace(ops, T, D, F) bytes, 256-byte aligned. */
GEMM_API size_t gemm_gated_ffn_workspace(gemm_ops_t ops, int64_t T, int64_t D, int64_t F);
GEMM_API gemm_status_t gemm_gated_ffn(gemm_ops_t ops, const void* x, int64_t ldx, const void* w_in,
                                      int64_t ldw_in, const void* w_down, int64_t ldw_down, void* y,
                                      int64_t ldy, void* gu, void* workspace, size_t workspace_bytes,
                                      int64_t T, int64_t D, int64_t F, gemm_act_t act,
                                      gemm_dtype_t dtype, void* stream);

/* Its gradients, given dy and the g and u that gemm_gated_ffn kept:
 *
 *     dh = dy Wd,  dg = dh u act'(g),  du = dh act(g),  h = act(g) u
 *     dx = dg Wg + du Wu,  dw_in = [dg du]^T x,  dw_down = dy^T h
 *
 *   dy : [T, D];  dx : [T, D];  dw_in : [2 F, D] and dw_down : [D, F], contiguous
 * dg, du and h are rounded to 16 bits as operands; relu's slope at 0 is 0.
 * Gradients are written, not accumulated; T == 0 gives zero dw_in and dw_down.
 * Rules as above. */
GEMM_API size_t gemm_gated_ffn_backward_workspace(gemm_ops_t ops, int64_t T, int64_t D, int64_t F);
GEMM_API gemm_status_t gemm_gated_ffn_backward(
    gemm_ops_t ops, const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w_in,
    int64_t ldw_in, const void* w_down, int64_t ldw_down, const void* gu, void* dx, int64_t lddx,
    void* dw_in, void* dw_down, void* workspace, size_t workspace_bytes, int64_t T, int64_t D,
    int64_t F, gemm_act_t act, gemm_dtype_t dtype, void* stream);

/* y = x W^T from 4-bit weights:  W[n, k] = scales[n, k / G] (q[n, k] - zeros[n, k / G]).
 *
 *   x      : [T, K], rows ldx apart;  y : [T, N], rows ldy apart
 *   codes  : [N, K / 2] bytes, contiguous: q of column 2j in the low half of
 *            byte j, of column 2j + 1 in the high half
 *   scales : [N, K / G] 16-bit, contiguous
 *   zeros  : [N, K / G] bytes 0 .. 15, or NULL for 8 everywhere
 *   group  : G, a power of two from 32 on that divides K
 * Made for few tokens: the weights are read once for every 16, and T is at most
 * 8 * 65535.  x and codes 16-byte aligned, ldx a multiple of 8
 * (GEMM_ERR_ALIGNMENT); ldy and the alignment of N are free; K is at most 2^28.
 * A group's sum of x (O + q - (O + zero)), O = 64 (fp16) or 128 (bf16), and its
 * product with the scale are fp32; the products x (O + q) are exact.  A sum that
 * does not come out finite so (an infinite x, or one whose products with O + q
 * overflow) is taken again, product by product (1 ms for 8192 x 8192): infinities
 * and NaN go where the formula puts them.
 * workspace: gemm_w4_workspace(ops, T, N, K, gated) bytes (none for most
 * shapes), 256-byte aligned. */
GEMM_API size_t gemm_w4_workspace(gemm_ops_t ops, int64_t T, int64_t N, int64_t K, int32_t gated);
GEMM_API gemm_status_t gemm_w4_linear(gemm_ops_t ops, const void* x, int64_t ldx, const void* codes,
                                      const void* scales, const void* zeros, void* y, int64_t ldy,
                                      void* workspace, size_t workspace_bytes, int64_t T, int64_t N, int64_t K, int64_t group,
                                      gemm_dtype_t dtype, void* stream);
/* y = act(x Wg^T) * (x Wu^T), W of 2 N rows (gate rows, then up rows). */
GEMM_API gemm_status_t gemm_w4_gated(gemm_ops_t ops, const void* x, int64_t ldx, const void* codes,
                                     const void* scales, const void* zeros, void* y, int64_t ldy,
                                     void* workspace, size_t workspace_bytes, int64_t T, int64_t N, int64_t K, int64_t group, gemm_act_t act,
                                     gemm_dtype_t dtype, void* stream);

/* The orthogonalised update: `steps` steps of an odd polynomial that drives
 * every singular value of m / (|m| + eps) (Frobenius norm) towards 1,
 *
 *     X <- a X + (b P + c P^2) X,   P = X X^T   (P = X^T X from the right
 *                                   when M > N: the same X)
 *
 * on `batch` matrices of M x N.
 *   m, out   : rows ldm / ldo apart, matrices stride_m / stride_o apart
 *              (elements), free and without alignment rules; batch <= 65535
 *   in_dtype, out_dtype : GEMM_F16, GEMM_BF16 or GEMM_F32
 *   coeffs   : a, b, c
 * X, P and b P + c P^2 are held to 22 bits, as the sum of two fp16 numbers
 * scaled by powers of two, and products of them are summed in fp32: rounding
 * them to one 16-bit number costs 1e-3 to 1e-2 of the result, since small
 * singular values grow by up to a^steps.  Their entries must stay below 8,
 * 32 and 64 (any coefficients that keep singular values below 2.8 and
 * |b| s^2 + |c| s^4 below 64); larger ones end in infinities and NaN.  Entries of
 * X below 2^-16 are held to 2^-38 instead.  The sum of squares is fp32: |m| must
 * be below 2^63, and above 2^-63 where eps is 0.  A matrix of a batch gets the
 * bits it gets by itself.
 * workspace: gemm_orthogonalize_workspace(ops, batch, M, N) bytes, 256-byte
 * aligned. */
GEMM_API size_t gemm_orthogonalize_workspace(gemm_ops_t ops, int64_t batch, int64_t M, int64_t N);
GEMM_API gemm_status_t gemm_orthogonalize(gemm_ops_t ops, const void* m, int64_t ldm, int64_t stride_m,
                                          void* out, int64_t ldo, int64_t stride_o, void* workspace,
                                          size_t workspace_bytes, int64_t batch, int64_t M, int64_t N,
                                          int32_t steps, const float coeffs[3], float eps,
                                          gemm_dtype_t in_dtype, gemm_dtype_t out_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_GEMM_OPS_H_ */
