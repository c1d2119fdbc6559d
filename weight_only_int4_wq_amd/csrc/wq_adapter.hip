// Low-rank adapters beside a quantized layer, forward and backward
// (wq_adapter.h).
#include "wq_adapter_common.h"

namespace {

using wq::Drop;

__device__ __forceinline__ int slot_of(const int32_t* slots, int m, int L) {
    const int s = slots ? slots[m] : 0;
    return unsigned(s) < unsigned(L) ? s : -1;
}

__device__ __forceinline__ float dropped(const Drop& d, uint64_t stream, uint64_t at, float v) {
    if (d.t == 0) return v;
    return wq::kept(wq::philox(at >> 3, stream, d.key0, d.key1), int(at & 7), d.t) ? v * d.keep : 0.f;
}

// h[m][r] = sum over c of dropout(src[m][c]) * w[slot][r][c]: a wavefront each.
__global__ __launch_bounds__(64) void shrink_kernel(const uint16_t* src, const uint16_t* w, const int32_t* slots,
                                                    Drop d, float* h, int R, int L, int C, int64_t first) {
    const int64_t q = first + blockIdx.x;
    const int m = int(q / R), r = int(q - int64_t(m) * R), a = slot_of(slots, m, L);
    float v = 0.f;
    if (a >= 0) {
        const uint64_t stream = wq::drop_stream(d);
        const uint16_t* row = w + (size_t(a) * R + r) * C;
        for (int c = threadIdx.x; c < C; c += 64)
            v += dropped(d, stream, uint64_t(m) * C + c, wq::h2f(src[size_t(m) * C + c])) * wq::h2f(row[c]);
    }
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    if (threadIdx.x == 0) h[q] = v;
}

// out[m][c] = add[m][c] + dropout'(s * sum over r of h[m][r] * w[slot][r][c])
__global__ __launch_bounds__(256) void expand_kernel(const float* h, const uint16_t* w, const float* scales,
                                                     const int32_t* slots, Drop d, const uint16_t* add, uint16_t* out,
                                                     int R, int L, int C, int64_t n, int64_t first) {
    const int64_t q = first + int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (q >= n) return;
    const int m = int(q / C), c = int(q - int64_t(m) * C), a = slot_of(slots, m, L);
    float v = 0.f;
    if (a >= 0) {
        for (int r = 0; r < R; ++r) v += h[size_t(m) * R + r] * wq::h2f(w[(size_t(a) * R + r) * C + c]);
        v = dropped(d, wq::drop_stream(d), uint64_t(q), v * scales[a]);
    }
    out[q] = wq::f2h(add ? wq::h2f(add[q]) + v : v);
}

// dw[a][r][c] = s * sum over a's rows of h[m][r] * dropout(src[m][c])
__global__ __launch_bounds__(256) void outer_kernel(const float* h, const uint16_t* src, const float* scales,
                                                    const int32_t* slots, Drop d, float* dw, int M, int R, int L,
                                                    int C, int64_t n, int64_t first) {
    const int64_t q = first + int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (q >= n) return;
    const int64_t ar = q / C;
    const int c = int(q - ar * C), a = int(ar / R), r = int(ar - int64_t(a) * R);
    const uint64_t stream = wq::drop_stream(d);
    float v = 0.f;
    for (int m = 0; m < M; ++m)
        if (slot_of(slots, m, L) == a)
            v += h[size_t(m) * R + r] * dropped(d, stream, uint64_t(m) * C + c, wq::h2f(src[size_t(m) * C + c]));
    dw[q] = M ? v * scales[a] : 0.f;
}

template <class Launch>
wq_status pieces(int64_t total, int64_t threads, const Launch& launch) {
    const int64_t per = int64_t(wqh::kMaxBlocks) * threads;
    for (int64_t first = 0; first < total; first += per) {
        launch(unsigned((std::min(total - first, per) + threads - 1) / threads), first);
        const wq_status st = wqh::launch_status();
        if (st != WQ_OK) return st;
    }
    return WQ_OK;
}

wq_status shrink(const wqh::Adapters& a, const uint16_t* src, const uint16_t* w, const Drop& d, float* h, int C,
                 hipStream_t s) {
    return pieces(int64_t(a.M) * a.R, 1, [&](unsigned blocks, int64_t first) {
        shrink_kernel<<<blocks, 64, 0, s>>>(src, w, a.slots, d, h, a.R, a.L, C, first);
    });
}

wq_status expand(const wqh::Adapters& a, const float* h, const uint16_t* w, const Drop& d, const uint16_t* add,
                 uint16_t* out, int C, hipStream_t s) {
    return pieces(int64_t(a.M) * C, 256, [&](unsigned blocks, int64_t first) {
        expand_kernel<<<blocks, 256, 0, s>>>(h, w, a.scales, a.slots, d, add, out, a.R, a.L, C, int64_t(a.M) * C,
                                             first);
    });
}

wq_status outer(const wqh::Adapters& a, const float* h, const uint16_t* src, const Drop& d, float* dw, int C,
                hipStream_t s) {
    const int64_t n = int64_t(a.L) * a.R * C;
    return pieces(n, 256, [&](unsigned blocks, int64_t first) {
        outer_kernel<<<blocks, 256, 0, s>>>(h, src, a.scales, a.slots, d, dw, a.M, a.R, a.L, C, n, first);
    });
}

constexpr Drop kNoDrop{0, 1.f, 0, 0, 0, nullptr};

}  // namespace

namespace wqh {

size_t adapters_workspace(int M, int, int, int R, int) { return size_t(M) * R * 4; }

wq_status adapters_forward(const Adapters& a, const uint16_t* x, const uint16_t* down, const uint16_t* up,
                           const uint16_t* base, uint16_t* y, float* hidden, int N, int K, void* ws, hipStream_t s) {
    float* h = hidden ? hidden : static_cast<float*>(ws);
    const wq_status st = shrink(a, x, down, a.drop, h, K, s);
    return st != WQ_OK ? st : expand(a, h, up, kNoDrop, base, y, N, s);
}

size_t adapters_backward_workspace(int M, int, int, int R, int) { return size_t(M) * R * 4; }

wq_status adapters_backward(const Adapters& a, const uint16_t* dy, const uint16_t* x, const float* hidden,
                            const uint16_t* down, const uint16_t* up, const uint16_t* dx_add, uint16_t* dx,
                            float* ddown, float* dup, int N, int K, void* ws, hipStream_t s) {
    float* dh = static_cast<float*>(ws);
    wq_status st = WQ_OK;
    if (a.M) st = shrink(a, dy, up, kNoDrop, dh, N, s);
    if (st == WQ_OK && dx) st = expand(a, dh, down, a.drop, dx_add, dx, K, s);
    if (st == WQ_OK && ddown) st = outer(a, dh, x, a.drop, ddown, K, s);
    if (st == WQ_OK && dup) st = outer(a, hidden, dy, kNoDrop, dup, N, s);
    return st;
}

}  // namespace wqh
