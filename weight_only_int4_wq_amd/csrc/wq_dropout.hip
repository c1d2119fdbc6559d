// Dropout from the counter-based generator (wq_adapter.h): elementwise.
#include "wq_adapter_common.h"

namespace {

// Eight elements share one block of the generator; a thread takes G such eights
// a block's width apart, all loads first.  Bound by memory: 8191 x 11005 elements
// 64 us (5.6 TB/s), 2048 x 4096 with a residual 9.2 (5.4 TB/s, from the last-level
// cache in part); one eight to a thread and 2-byte accesses took 175 and 31.  Up to
// 4 million elements one eight to a thread fills more units: 64 x 4096 2.5 us.
template <int G, bool RESIDUAL>
__global__ __launch_bounds__(256) void dropout_kernel(const uint16_t* x, const uint16_t* residual, wq::Drop d,
                                                      uint16_t* y, int64_t n, int64_t first) {
    const int64_t b0 = (first + blockIdx.x) * (256 * G);   // the block's first eight
    const uint64_t stream = wq::drop_stream(d);
    auto eight = [&](float (&v)[8], const float* r, int64_t at) {
        const wq::u4 w = wq::philox(uint64_t(at), stream, d.key0, d.key1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = wq::kept(w, i, d.t) ? v[i] * d.keep : 0.f;
            if (RESIDUAL) v[i] += r[i];
        }
    };
    if ((b0 + 256 * G) * 8 <= n) {
        wq::u4 a[G], r[G];
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const int64_t at = (b0 + 256 * k + threadIdx.x) * 8;
            a[k] = *reinterpret_cast<const wq::u4*>(x + at);
            if (RESIDUAL) r[k] = *reinterpret_cast<const wq::u4*>(residual + at);
        }
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const int64_t at = b0 + 256 * k + threadIdx.x;
            float v[8], f[8];
            wq::load_h<8>(reinterpret_cast<const uint16_t*>(&a[k]), v);
            if (RESIDUAL) wq::load_h<8>(reinterpret_cast<const uint16_t*>(&r[k]), f);
            eight(v, f, at);
            wq::store_h<8>(y + at * 8, v);
        }
        return;
    }
    for (int k = 0; k < G; ++k) {   // the last block
        const int64_t at = b0 + 256 * k + threadIdx.x;
        const int64_t left = n - at * 8;
        if (left <= 0) return;
        float v[8], f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = i < left ? wq::h2f(x[at * 8 + i]) : 0.f;
            f[i] = RESIDUAL && i < left ? wq::h2f(residual[at * 8 + i]) : 0.f;
        }
        eight(v, f, at);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) y[at * 8 + i] = wq::f2h(v[i]);
    }
}

}  // namespace

namespace wqh {

wq_status dropout(const uint16_t* x, const uint16_t* residual, const wq::Drop& d, uint16_t* y, int64_t n,
                  hipStream_t s) {
    const int64_t groups = (n + 7) / 8;
    auto run = [&](auto g) {
        constexpr int G = decltype(g)::value;
        const int64_t blocks = (groups + 256 * G - 1) / (256 * G);
        for (int64_t first = 0; first < blocks; first += kMaxBlocks) {
            const unsigned now = unsigned(std::min<int64_t>(blocks - first, kMaxBlocks));
            if (residual)
                dropout_kernel<G, true><<<now, 256, 0, s>>>(x, residual, d, y, n, first);
            else
                dropout_kernel<G, false><<<now, 256, 0, s>>>(x, residual, d, y, n, first);
            const wq_status st = launch_status();
            if (st != WQ_OK) return st;
        }
        return WQ_OK;
    };
    return groups <= 256 * 2048 ? run(std::integral_constant<int, 1>{}) : run(std::integral_constant<int, 4>{});
}

}  // namespace wqh
