/*
 * wq_block.h - the products of a quantized feed-forward block, forward and
 * backward, on libwq's packed weights (same library and conventions as wq.h).
 *
 * wq_linear_act       y = act(x . W^T + bias) + residual
 * wq_gated            h = act(x . Wg^T + bg) * (x . Wu^T + bu)
 * and their backward passes with respect to the activations, the bias and
 * the residual (the packed weights are frozen: they have no gradient).
 * Fusing a block's operations into single kernels saves launches and
 * intermediate tensors ("AutoAWQ vs The Stack v2", paragraph on fused
 * attention and transformer blocks); adapters trained on frozen quantized
 * weights need the gradient through them ("AutoGPTQ vs The Stack v2",
 * paragraph on LoRA and PEFT).
 *
 * W [N][K] = fp16((q - z) * s), exactly the weights wq_dequant writes, in
 * every kernel behind these entry points: forward and backward, one token or
 * many, see the same weights.  Products accumulate in fp32.
 *
 * Conventions beyond wq.h's:
 *  - every array is 16-byte aligned, except scales and zeros;
 *  - K and the number of weight rows are at most 2^22, M at most 2^30, and
 *    the outputs fewer than 2^24 tiles of 256 rows by 256 weight rows
 *    (backward: by 256 channels) (WQ_ERR_ARG past that);
 *  - zero-points are below 2^bits (8-bit: any byte);
 *  - rows are independent: row m of an output depends on row m of the inputs
 *    only, so rows that hold padding, infinities or NaN leave the others as
 *    they are;
 *  - with act-order (perm != NULL) x and dx are in original channel order,
 *    as for wq_linear.  perm must be a permutation of 0 .. K-1;
 *  - outputs and the workspace share no memory with inputs or each other
 *    (WQ_ERR_ARG), except that y may be residual and dx may be dx_add, whole;
 *  - sums run in a fixed order: the same call gives the same bits, whatever
 *    the workspace holds.  A call with less optional workspace, or with
 *    another M, may add in another order;
 *  - workspace: device memory of at least the bytes the matching
 *    *_workspace_size returns, 16-byte aligned, or NULL when that is 0.
 *    Less is accepted down to the part that cannot be left out (see each
 *    call); WQ_ERR_ARG below it.  Calls that share a workspace must be
 *    ordered on one stream, captured graphs among them;
 *  - all calls are asynchronous, allocate nothing and can be captured into a
 *    graph.  The current device must be the stream's device.
 */
#ifndef WQ_BLOCK_H
#define WQ_BLOCK_H

#include "wq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations.  Both limits are taken at infinities: silu(-inf) = 0. */
typedef enum {
    WQ_ACT_NONE = 0,      /* v                                        */
    WQ_ACT_RELU = 1,      /* max(v, 0), derivative 0 at 0             */
    WQ_ACT_GELU = 2,      /* v * Phi(v), Phi the normal distribution  */
    WQ_ACT_GELU_TANH = 3, /* v / 2 * (1 + tanh(sqrt(2 / pi) * (v + 0.044715 v^3))) */
    WQ_ACT_SILU = 4       /* v / (1 + e^-v)                           */
} wq_act;

/* z = x . W^T + bias in fp32; y = fp16(act(z) + residual), rounded once;
 * preact = fp16(z) for the backward pass.
 * x fp16 [M][K]; bias fp16 [N] (nullable); residual fp16 [M][N] (nullable,
 * may be y itself: an update in place); y fp16 [M][N]; preact fp16 [M][N]
 * (nullable).  act: a wq_act.  M >= 0, N >= 0 (0: nothing is done).
 * The workspace part that cannot be left out: act-order's gathered
 * activations, M*K*2 bytes rounded up to 256; the rest holds fp32 partial
 * sums of a K split (without it K is not split across blocks).
 * WQ_ERR_ARG: null or misaligned pointers, bad sizes or activation, a short
 * workspace; WQ_ERR_UNSUPPORTED: other bit widths. */
wq_status wq_linear_act(const uint16_t* x, const uint32_t* packed, const uint16_t* scales, const uint8_t* zeros,
                        const int32_t* perm, const uint16_t* bias, const uint16_t* residual, int32_t act,
                        uint16_t* y, uint16_t* preact, int32_t M, int32_t N, int32_t K, int32_t bits,
                        int32_t group_size, void* workspace, size_t workspace_bytes, void* stream);
size_t wq_linear_act_workspace_size(int32_t M, int32_t N, int32_t K, int32_t bits, int32_t has_perm);

/* Gate and up projections, activation and product in one kernel.  The 2 I
 * rows of packed / scales / zeros / bias are the gate projection (rows
 * 0 .. I-1) stacked over the up projection (rows I .. 2I-1), as for
 * wq_gemv_silu_mul, for any M and activation:
 *   g = x . Wg^T + bg, u = x . Wu^T + bu in fp32;  h = fp16(act(g) * u);
 * preact fp16 [M][2 I] = (fp16(g), fp16(u)) side by side (nullable).
 * h fp16 [M][I].  Otherwise as wq_linear_act. */
wq_status wq_gated(const uint16_t* x, const uint32_t* packed, const uint16_t* scales, const uint8_t* zeros,
                   const int32_t* perm, const uint16_t* bias, int32_t act, uint16_t* h, uint16_t* preact, int32_t M,
                   int32_t I, int32_t K, int32_t bits, int32_t group_size, void* workspace, size_t workspace_bytes,
                   void* stream);
size_t wq_gated_workspace_size(int32_t M, int32_t I, int32_t K, int32_t bits, int32_t has_perm);

/* Backward of wq_linear_act for dy fp16 [M][N]:
 *   dz = fp16(dy * act'(preact))   (dy itself for WQ_ACT_NONE),
 *   dx = fp16(dz . W + dx_add),    dbias[n] = sum over m of dy * act'(preact).
 * preact fp16 [M][N], required unless act is WQ_ACT_NONE; dx_add fp16 [M][K]
 * (nullable, may be dx itself); dx fp16 [M][K]; dz fp16 [M][N] (nullable: the
 * gradient that adapters on this layer take); dbias fp32 [N]
 * (nullable; fp32 because a sum over thousands of rows leaves fp16's
 * range).  The residual's gradient is dy.  dz enters the product in fp16, as
 * the matrix cores take it: where it leaves fp16's range it is infinite, and
 * that row of dx infinite or NaN.  With M = 0 dbias is zero; with N = 0 dx is
 * dx_add or zero.
 * The workspace part that cannot be left out: dz rows padded to a multiple of
 * 8 when dz is NULL and the activation is not WQ_ACT_NONE, or when N is no
 * multiple of 8; dbias's partial sums when dbias is given; with act-order
 * fp32 dx, its rows rounded up to 64 and its columns to 256.  The rest holds
 * partial sums of an N split. */
wq_status wq_linear_act_backward(const uint16_t* dy, const uint16_t* preact, int32_t act, const uint32_t* packed,
                                 const uint16_t* scales, const uint8_t* zeros, const int32_t* perm,
                                 const uint16_t* dx_add, uint16_t* dx, uint16_t* dz, float* dbias, int32_t M,
                                 int32_t N, int32_t K, int32_t bits, int32_t group_size, void* workspace,
                                 size_t workspace_bytes, void* stream);
size_t wq_linear_act_backward_workspace_size(int32_t M, int32_t N, int32_t K, int32_t bits, int32_t has_perm);

/* Backward of wq_gated for dh fp16 [M][I] and the kept preact fp16 [M][2 I]
 * (required for every activation):
 *   dg = fp16(dh * u * act'(g)), du = fp16(dh * act(g)), dz = (dg, du),
 *   dx = fp16(dz . W + dx_add),  dbias fp32 [2 I] = column sums.
 * dz fp16 [M][2 I].  Otherwise as wq_linear_act_backward. */
wq_status wq_gated_backward(const uint16_t* dh, const uint16_t* preact, int32_t act, const uint32_t* packed,
                            const uint16_t* scales, const uint8_t* zeros, const int32_t* perm,
                            const uint16_t* dx_add, uint16_t* dx, uint16_t* dz, float* dbias, int32_t M, int32_t I,
                            int32_t K, int32_t bits, int32_t group_size, void* workspace, size_t workspace_bytes,
                            void* stream);
size_t wq_gated_backward_workspace_size(int32_t M, int32_t I, int32_t K, int32_t bits, int32_t has_perm);

#ifdef __cplusplus
}
#endif

#endif /* WQ_BLOCK_H */
