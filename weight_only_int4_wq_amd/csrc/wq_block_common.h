// Shared parts of the feed-forward block's kernels (wq_block.h): activations
// and their derivatives, the forward epilogue, fp16 vector accesses.
#pragma once

#include "../../include/wq_block.h"
#include "wq_gemm_common.h"

namespace wq {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float h2f(uint16_t v) { return float(__builtin_bit_cast(_Float16, v)); }
__device__ __forceinline__ uint16_t f2h(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

// V fp16 values at p as floats, and back with one rounding each.  V > 1 needs
// p aligned to 2 V bytes.
template <int V>
struct Half {
    uint16_t e[V];
};
template <int V>
__device__ __forceinline__ void load_h(const uint16_t* p, float (&v)[V]) {
    Half<V> h;
    __builtin_memcpy(&h, __builtin_assume_aligned(p, 2 * V), 2 * V);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = h2f(h.e[i]);
}
template <int V>
__device__ __forceinline__ void store_h(uint16_t* p, const float (&v)[V]) {
    Half<V> h;
#pragma unroll
    for (int i = 0; i < V; ++i) h.e[i] = f2h(v[i]);
    __builtin_memcpy(__builtin_assume_aligned(p, 2 * V), &h, 2 * V);
}

// 1 / (1 + e^-v).  For v below -88 e^-v overflows to infinity and the result
// is 0, its limit to fp32's accuracy.
__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + __expf(-v)); }

constexpr float kSqrtHalf = 0.70710678118654752f;     // sqrt(1 / 2)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;   // 1 / sqrt(2 pi)
constexpr float kTanhScale = 0.79788456080286536f;    // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// act(v).  gelu as v/2 erfc(-v / sqrt 2) and gelu_tanh as v sigmoid(2 u)
// (the same functions): neither cancels for negative v.  Arguments are held
// above -100, where every one of them is 0 to fp32's accuracy, so that -inf
// gives the limit 0 and not inf * 0; NaN passes through the comparison.
__device__ __forceinline__ float act_value(float v, int kind) {
    switch (kind) {
        case WQ_ACT_RELU: return v < 0.f ? 0.f : v;
        case WQ_ACT_GELU: {
            const float c = v < -100.f ? -100.f : v;
            return 0.5f * c * erfcf(-kSqrtHalf * c);
        }
        case WQ_ACT_GELU_TANH: {
            const float c = v < -100.f ? -100.f : v;
            return c * sigmoid(2.f * kTanhScale * __builtin_fmaf(kTanhCubic * c * c, c, c));
        }
        case WQ_ACT_SILU: {
            const float c = v < -100.f ? -100.f : v;
            return c * sigmoid(c);
        }
        default: return v;
    }
}

// act(v) and act'(v), v held within +-100 for the derivative (it is 0 or 1
// there to fp32's accuracy).
__device__ __forceinline__ float act_slope(float v, int kind, float& value) {
    value = act_value(v, kind);
    const float c = v < -100.f ? -100.f : v > 100.f ? 100.f : v;
    switch (kind) {
        case WQ_ACT_RELU: return v > 0.f ? 1.f : v != v ? v : 0.f;
        case WQ_ACT_GELU:
            return __builtin_fmaf(c * kInvSqrt2Pi, __expf(-0.5f * c * c), 0.5f * erfcf(-kSqrtHalf * c));
        case WQ_ACT_GELU_TANH: {
            const float t = sigmoid(2.f * kTanhScale * __builtin_fmaf(kTanhCubic * c * c, c, c));
            const float du = 2.f * kTanhScale * __builtin_fmaf(3.f * kTanhCubic * c, c, 1.f);
            return __builtin_fmaf(c * t * (1.f - t), du, t);
        }
        case WQ_ACT_SILU: {
            const float t = sigmoid(c);
            return t * __builtin_fmaf(c, 1.f - t, 1.f);
        }
        default: return 1.f;
    }
}

// What follows the forward product.  The linear layer has `out` output
// columns of the same number of weight rows, the gated block `out` = I
// columns of 2 I weight rows.
struct Epilogue {
    const uint16_t* bias;      // fp16 [rows], nullable
    const uint16_t* residual;  // fp16 [M][out], nullable, may be y
    uint16_t* y;               // fp16 [M][out]
    uint16_t* preact;          // fp16 [M][rows], nullable
    int out;
    int act;
};

// V outputs of one row from column col on: a = the fp32 products (gated: the
// gate's), u = the up projection's.  V > 1 needs out and col to be multiples
// of V.
template <bool GATED, int V>
__device__ __forceinline__ void finish(const Epilogue& e, int row, int col, float (&a)[V], float (&u)[V]) {
    const size_t at = size_t(row) * e.out + col;
    if (e.bias) {
        float b[V];
        load_h<V>(e.bias + col, b);
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] += b[i];
        if constexpr (GATED) {
            load_h<V>(e.bias + e.out + col, b);
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] += b[i];
        }
    }
    if (e.preact) {
        uint16_t* p = e.preact + (GATED ? 2 * (at - col) + col : at);
        store_h<V>(p, a);
        if constexpr (GATED) store_h<V>(p + e.out, u);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        a[i] = act_value(a[i], e.act);
        if constexpr (GATED) a[i] *= u[i];
    }
    if constexpr (!GATED) {
        if (e.residual) {
            float r[V];
            load_h<V>(e.residual + at, r);
#pragma unroll
            for (int i = 0; i < V; ++i) a[i] += r[i];
        }
    }
    store_h<V>(e.y + at, a);
}

}  // namespace wq

namespace wqh {

// One forward product of the block: x [M][K] in packed channel order, `rows`
// weight rows (gated: 2 * e.out).
struct BlockFwd {
    const uint16_t* x;
    const uint32_t* packed;
    const uint16_t* scales;
    const uint8_t* zeros;
    int M, rows, K, bits, gs;
    bool gated;
    wq::Epilogue e;
};

// Bytes of fp32 partial sums the product would like.
size_t block_fwd_part_bytes(int M, int rows, int K, int bits, bool gated);
wq_status block_fwd(const BlockFwd& p, float* part, size_t part_bytes, hipStream_t s);

// Small M (decode batches).
constexpr int kBlockSmallM = 32;
size_t block_small_part_bytes(int M, int rows, int K, int bits, bool gated);
wq_status block_small(const BlockFwd& p, float* part, size_t part_bytes, hipStream_t s);

// e applied to the sum over `splits` partial products [splits][M][rows].
wq_status block_finish(const wq::Epilogue& e, bool gated, const float* part, int splits, int M, hipStream_t s);

}  // namespace wqh
