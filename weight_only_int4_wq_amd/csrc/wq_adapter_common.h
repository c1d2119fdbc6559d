// Shared parts of the adapters' and dropout's kernels (wq_adapter.h).
#pragma once

#include "../../include/wq_adapter.h"
#include "wq_block_common.h"

namespace wq {

// Which elements dropout keeps.  t = 0: all of them.
struct Drop {
    uint32_t t;            // a half word below it drops the element
    float keep;            // 65536 / (65536 - t)
    uint32_t key0, key1;   // the seed
    uint64_t offset;
    const int64_t* step;   // added to offset; nullable
};

// The second half of the generator's counter: offset + *step.
__device__ __forceinline__ uint64_t drop_stream(const Drop& d) {
    return d.offset + (d.step ? uint64_t(*d.step) : 0u);
}

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
    return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// Philox4x32-10's output for the counters (n[i], stream).  Several at a time:
// a round's two products wait for the round before, and those of different
// counters do not.  The rounds are not unrolled, which would fill the
// instruction cache where a kernel's code runs once per wavefront.
template <int N>
__device__ __forceinline__ void philox(const uint64_t (&n)[N], uint64_t stream, uint32_t k0, uint32_t k1, u4 (&w)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        w[i] = u4{uint32_t(n[i]), uint32_t(n[i] >> 32), uint32_t(stream), uint32_t(stream >> 32)};
#pragma unroll 1
    for (int r = 0; r < 10; ++r) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint64_t a = uint64_t(w[i][0]) * 0xD2511F53u, b = uint64_t(w[i][2]) * 0xCD9E8D57u;
            w[i] = u4{xor3(uint32_t(b >> 32), w[i][1], k0), uint32_t(b), xor3(uint32_t(a >> 32), w[i][3], k1),
                      uint32_t(a)};
        }
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}
__device__ __forceinline__ u4 philox(uint64_t n, uint64_t stream, uint32_t k0, uint32_t k1) {
    u4 w[1];
    philox<1>({n}, stream, k0, k1, w);
    return w[0];
}

// Whether element i of a block's eight is kept.
__device__ __forceinline__ bool kept(u4 w, int i, uint32_t t) {
    return (i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu) >= t;
}

typedef uint16_t us2 __attribute__((ext_vector_type(2)));

// All ones in the 16 bits of those of block n[i]'s eight elements that are kept
// (t > 0).
template <int N>
__device__ __forceinline__ void keep8(const uint64_t (&n)[N], const Drop& d, uint64_t stream, u4 (&w)[N]) {
    philox(n, stream, d.key0, d.key1, w);
    const us2 below{uint16_t(d.t - 1), uint16_t(d.t - 1)};
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = w[k][i];
            const us2 over = __builtin_elementwise_sub_sat(__builtin_bit_cast(us2, v), below);  // 0 below t
            w[k][i] = __builtin_bit_cast(uint32_t, us2(us2{0, 0} - __builtin_elementwise_min(over, us2{1, 1})));
        }
}

}  // namespace wq

namespace wqh {

// Sizes and operands of both adapter passes: src [M][C] . w[a]^T -> [M][R].
struct Adapters {
    const float* scales;
    const int32_t* slots;
    int M, R, L;
    wq::Drop drop;
};

size_t adapters_workspace(int M, int N, int K, int R, int L, bool dropping);
wq_status adapters_forward(const Adapters& a, const uint16_t* x, const uint16_t* down, const uint16_t* up,
                           const uint16_t* base, uint16_t* y, float* hidden, int N, int K, void* ws, hipStream_t s);
size_t adapters_backward_workspace(int M, int N, int K, int R, int L);
wq_status adapters_backward(const Adapters& a, const uint16_t* dy, const uint16_t* x, const float* hidden,
                            const uint16_t* down, const uint16_t* up, const uint16_t* dx_add, uint16_t* dx,
                            float* ddown, float* dup, int N, int K, void* ws, hipStream_t s);
wq_status dropout(const uint16_t* x, const uint16_t* residual, const wq::Drop& d, uint16_t* y, int64_t n,
                  hipStream_t s);

}  // namespace wqh
