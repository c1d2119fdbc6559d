/*
 * wq_adapter.h - low-rank adapters beside a quantized layer, and dropout
 * (same library and conventions as wq.h and wq_block.h).
 *
 * wq_adapters           y[m] = base[m] + s[a] * (x'[m] . down[a]^T) . up[a]
 * wq_adapters_backward  gradients of x, down and up
 * wq_dropout            y = (kept ? x / (1 - p) : 0) + residual; its own
 *                       backward pass on dy with the same numbers
 *
 * Row m takes adapter a = slots[m]; x' = dropout(x) where p > 0, else x.
 * The quantized layer's weights stay frozen and shared; each request brings
 * its own adapter, and adapters are what is trained on such a layer
 * ("AutoGPTQ vs The Stack v2", paragraph on LoRA and PEFT).
 *
 * Layouts:
 *  - x, dx, dx_add fp16 [M][K]; y, base, dy fp16 [M][N]; hidden fp32 [M][rank];
 *  - down fp16 [adapters][rank][K]; up fp16 [adapters][rank][N]: the second
 *    factor is stored transposed, so that both are read along their long
 *    side by either pass; ddown and dup are fp32 of the same shapes.
 *    Adapters of a lower rank than the pool's are filled with zeros;
 *  - scales fp32 [adapters], on the device;
 *  - slots int32 [M] in any order, or NULL: every row takes adapter 0.  A row
 *    whose slot is not in 0 .. adapters - 1 has no adapter: y is base (or
 *    zero), hidden zero, dx dx_add (or zero), and no gradient sees the row.
 *    Runs of neighbouring rows with one adapter are the fast case.
 * base may be y and dx_add may be dx (update in place); with neither given
 * the products stand alone.
 *
 * Dropout.  Elements of x are numbered in row-major order.  Eight at a time
 * share a block of the counter-based generator Philox4x32-10 (Salmon, Moraes,
 * Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011): its
 * counter is the eight's number (low, high word), then offset + *step modulo
 * 2^64 (low, high word), its key the seed (low, high word).  Element i of the
 * eight takes the low (i even) or high (i odd) half of output word i / 2, and
 * is kept where that is at least t = floor(65536 p + 1/2).  Kept elements are
 * multiplied by 65536 / (65536 - t), rounded to fp32; the others become +0
 * whatever they hold.  So p is taken in steps of 2^-16; 0 <= p < 1, and p
 * that rounds to 1 is refused.  The mask is never stored: a backward pass
 * makes it again from the same seed, offset and step.  step (int64 on the
 * device, nullable: 0) lets a captured graph draw another mask on every
 * replay: the caller advances it between the replays.
 *
 * Arithmetic: products accumulate in fp32 (whose rounding counts a subnormal
 * fp16 operand as 2^-14), and hidden keeps its 32 bits.  On
 * the way into the second product an element of it (of dh, of the hidden of a
 * backward call) is split into two fp16 numbers, after a power of two has
 * brought the largest one beside it into fp16's range: it is off by at most
 * 2^-22 of itself or 2^-38 of that largest one, whichever is more, and is zero
 * below 2^-39 of it.  Beside it, for y and dx, is its row; for ddown and dup its
 * column of 32 rows that follow one another among the adapter's: a row there that
 * is more than 2^16 times smaller than another has fewer than 22 bits.  y and
 * dx are rounded once.  Infinities and NaN in any operand give what the
 * products and sums of these numbers give them.
 *
 * Conventions: fp16 arrays, fp32 outputs and the workspace are 16-byte
 * aligned, slots and scales 4-byte, step 8-byte.  Outputs and the workspace
 * share no memory with inputs or each other, except as said.  Rows are
 * independent in y, hidden and dx.  Sums run in a fixed order: the same call
 * gives the same bits.  Calls are asynchronous, allocate nothing and can be
 * captured; calls that share a workspace must be ordered.  The current device
 * must be the stream's device.
 * Limits: M <= 2^30; N, K and adapters <= 2^22; 1 <= rank <= 128
 * (WQ_ERR_UNSUPPORTED above); K a multiple of 32, N any.
 */
#ifndef WQ_ADAPTER_H
#define WQ_ADAPTER_H

#include "wq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* hidden (nullable) receives x' . down^T for the backward pass, without the
 * scale.  M = 0: nothing is done.  workspace: at least
 * wq_adapters_workspace_size bytes (0 for small decode batches without
 * dropout: then it may be NULL).
 * WQ_ERR_ARG: null or misaligned pointers, bad sizes or p, overlaps, a short
 * workspace. */
wq_status wq_adapters(const uint16_t* x, const uint16_t* down, const uint16_t* up, const float* scales,
                      const int32_t* slots, const uint16_t* base, double p, uint64_t seed, uint64_t offset,
                      const int64_t* step, uint16_t* y, float* hidden, int32_t M, int32_t N, int32_t K, int32_t rank,
                      int32_t adapters, void* workspace, size_t workspace_bytes, void* stream);
/* has_dropout: whether p > 0; enough for both when set. */
size_t wq_adapters_workspace_size(int32_t M, int32_t N, int32_t K, int32_t rank, int32_t adapters,
                                  int32_t has_dropout);

/* For dy and the x, hidden and dropout numbers of the forward call:
 *   dh[m] = s[a] dy[m] . up[a]^T,  dx[m] = dropout'(dh[m] . down[a]) + dx_add[m],
 *   ddown[a] = sum over a's rows of dh[m]^T x'[m],
 *   dup[a] = s[a] * sum over a's rows of hidden[m]^T dy[m].
 * dx is nullable; ddown and dup are given together or both NULL, and x and
 * hidden may be NULL without them.  Adapters that no row takes get zero
 * gradients (all of them where M = 0).  base's gradient is dy. */
wq_status wq_adapters_backward(const uint16_t* dy, const uint16_t* x, const float* hidden, const uint16_t* down,
                               const uint16_t* up, const float* scales, const int32_t* slots, double p,
                               uint64_t seed, uint64_t offset, const int64_t* step, const uint16_t* dx_add,
                               uint16_t* dx, float* ddown, float* dup, int32_t M, int32_t N, int32_t K, int32_t rank,
                               int32_t adapters, void* workspace, size_t workspace_bytes, void* stream);
size_t wq_adapters_backward_workspace_size(int32_t M, int32_t N, int32_t K, int32_t rank, int32_t adapters);

/* x, residual (nullable) and y fp16 [n], 0 <= n < 2^62, rounded once.  y may
 * be x or residual.  The backward pass is the same call on dy without a
 * residual; the residual's gradient is dy. */
wq_status wq_dropout(const uint16_t* x, const uint16_t* residual, double p, uint64_t seed, uint64_t offset,
                     const int64_t* step, uint16_t* y, int64_t n, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WQ_ADAPTER_H */
