// Dropout from the counter-based generator (wq_adapter.h): elementwise.
#include "wq_adapter_common.h"

namespace {

// One thread to eight elements, which share one block of the generator.
__global__ __launch_bounds__(256) void dropout_kernel(const uint16_t* __restrict__ x,
                                                      const uint16_t* __restrict__ residual, wq::Drop d,
                                                      uint16_t* __restrict__ y, int64_t n, int64_t first) {
    const int64_t g = first + int64_t(blockIdx.x) * 256 + threadIdx.x, at = g * 8;
    if (at >= n) return;
    const wq::u4 w = wq::philox(uint64_t(g), wq::drop_stream(d), d.key0, d.key1);
    for (int i = 0; i < 8 && at + i < n; ++i) {
        float v = wq::kept(w, i, d.t) ? wq::h2f(x[at + i]) * d.keep : 0.f;
        if (residual) v += wq::h2f(residual[at + i]);
        y[at + i] = wq::f2h(v);
    }
}

}  // namespace

namespace wqh {

wq_status dropout(const uint16_t* x, const uint16_t* residual, const wq::Drop& d, uint16_t* y, int64_t n,
                  hipStream_t s) {
    const int64_t per = int64_t(kMaxBlocks) * 256, groups = (n + 7) / 8;
    for (int64_t first = 0; first < groups; first += per) {
        const unsigned blocks = unsigned((std::min(groups - first, per) + 255) / 256);
        dropout_kernel<<<blocks, 256, 0, s>>>(x, residual, d, y, n, first);
        const wq_status st = launch_status();
        if (st != WQ_OK) return st;
    }
    return WQ_OK;
}

}  // namespace wqh
