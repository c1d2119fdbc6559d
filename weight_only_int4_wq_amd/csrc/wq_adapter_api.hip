// Entry points of wq_adapter.h: argument checks and workspace sizes.
#include <initializer_list>

#include "wq_adapter_common.h"

namespace {

constexpr int kMaxWidth = 1 << 22, kMaxRank = 128;

bool sizes_ok(int M, int N, int K, int rank, int adapters) {
    return M >= 0 && M <= (1 << 30) && N > 0 && N <= kMaxWidth && K > 0 && K % 32 == 0 && K <= kMaxWidth && rank > 0 &&
           adapters > 0 && adapters <= kMaxWidth;
}

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// An array of the caller's, empty when it is null.
struct Bytes {
    uintptr_t at;
    size_t n;
    Bytes(const void* p, size_t bytes) : at(reinterpret_cast<uintptr_t>(p)), n(p ? bytes : 0) {}
    bool overlaps(const Bytes& o) const { return n && o.n && (at <= o.at ? o.at - at < n : at - o.at < o.n); }
};

// Whether something that a call writes shares memory with something that it
// reads or with something else that it writes.
bool clash(std::initializer_list<Bytes> written, std::initializer_list<Bytes> read) {
    for (auto w = written.begin(); w != written.end(); ++w) {
        for (const Bytes& r : read)
            if (w->overlaps(r)) return true;
        for (auto o = w + 1; o != written.end(); ++o)
            if (w->overlaps(*o)) return true;
    }
    return false;
}

// False for p outside [0, 1), NaN, or so near to 1 that nothing is kept.
bool drop_of(double p, uint64_t seed, uint64_t offset, const int64_t* step, wq::Drop& d) {
    if (!(p >= 0.0 && p < 1.0) || !aligned(step, 8)) return false;
    d.t = uint32_t(p * 65536.0 + 0.5);
    if (d.t > 65535u) return false;
    d.keep = float(65536.0 / double(65536u - d.t));
    d.key0 = uint32_t(seed);
    d.key1 = uint32_t(seed >> 32);
    d.offset = offset;
    d.step = step;
    return true;
}

bool all_aligned16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!wqh::aligned16(p)) return false;
    return true;
}

}  // namespace

extern "C" wq_status wq_adapters(const uint16_t* x, const uint16_t* down, const uint16_t* up, const float* scales,
                                 const int32_t* slots, const uint16_t* base, double p, uint64_t seed, uint64_t offset,
                                 const int64_t* step, uint16_t* y, float* hidden, int32_t M, int32_t N, int32_t K,
                                 int32_t rank, int32_t adapters, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    wqh::Adapters a{scales, slots, M, rank, adapters, {}};
    if (!sizes_ok(M, N, K, rank, adapters) || !drop_of(p, seed, offset, step, a.drop)) return WQ_ERR_ARG;
    if (!all_aligned16({x, down, up, base, y, hidden, workspace}) || !aligned(scales, 4) || !aligned(slots, 4))
        return WQ_ERR_ARG;
    if (rank > kMaxRank) return WQ_ERR_UNSUPPORTED;
    if (M == 0) return WQ_OK;
    if (!x || !down || !up || !scales || !y) return WQ_ERR_ARG;
    const size_t need = wqh::adapters_workspace(M, N, K, rank, adapters, a.drop.t != 0);
    if (need > (workspace ? workspace_bytes : 0)) return WQ_ERR_ARG;
    const size_t ny = size_t(M) * N * 2, pool = size_t(adapters) * rank * 2;
    if (clash({{y, ny}, {hidden, size_t(M) * rank * 4}, {workspace, workspace_bytes}},
              {{x, size_t(M) * K * 2}, {down, pool * K}, {up, pool * N}, {scales, size_t(adapters) * 4},
               {slots, size_t(M) * 4}, {step, 8}, {base == y ? nullptr : base, ny}}))
        return WQ_ERR_ARG;
    return wqh::adapters_forward(a, x, down, up, base, y, hidden, N, K, workspace, static_cast<hipStream_t>(stream));
}

extern "C" size_t wq_adapters_workspace_size(int32_t M, int32_t N, int32_t K, int32_t rank, int32_t adapters,
                                             int32_t has_dropout) {
    return sizes_ok(M, N, K, rank, adapters) && rank <= kMaxRank && M > 0
               ? wqh::adapters_workspace(M, N, K, rank, adapters, has_dropout != 0) : 0;
}

extern "C" wq_status wq_adapters_backward(const uint16_t* dy, const uint16_t* x, const float* hidden,
                                          const uint16_t* down, const uint16_t* up, const float* scales,
                                          const int32_t* slots, double p, uint64_t seed, uint64_t offset,
                                          const int64_t* step, const uint16_t* dx_add, uint16_t* dx, float* ddown,
                                          float* dup, int32_t M, int32_t N, int32_t K, int32_t rank, int32_t adapters,
                                          void* workspace, size_t workspace_bytes, void* stream) {
    wqh::Adapters a{scales, slots, M, rank, adapters, {}};
    if (!sizes_ok(M, N, K, rank, adapters) || !drop_of(p, seed, offset, step, a.drop)) return WQ_ERR_ARG;
    if (!all_aligned16({dy, x, hidden, down, up, dx_add, dx, ddown, dup, workspace}) || !aligned(scales, 4) ||
        !aligned(slots, 4))
        return WQ_ERR_ARG;
    if (rank > kMaxRank) return WQ_ERR_UNSUPPORTED;
    if (!ddown != !dup) return WQ_ERR_ARG;
    const size_t pool = size_t(adapters) * rank;
    if (M == 0) {
        if (!ddown) return WQ_OK;
        if (clash({{ddown, pool * K * 4}, {dup, pool * N * 4}}, {})) return WQ_ERR_ARG;
        return wqh::adapters_backward(a, dy, x, hidden, down, up, dx_add, nullptr, ddown, dup, N, K, workspace,
                                      static_cast<hipStream_t>(stream));
    }
    if (!dx && !ddown) return WQ_OK;
    if (!dy || !up || !scales || (dx && !down) || (ddown && (!x || !hidden))) return WQ_ERR_ARG;
    const size_t need = wqh::adapters_backward_workspace(M, N, K, rank, adapters);
    if (need > (workspace ? workspace_bytes : 0)) return WQ_ERR_ARG;
    const size_t nx = size_t(M) * K * 2;
    if (clash({{dx, nx}, {ddown, pool * K * 4}, {dup, pool * N * 4}, {workspace, workspace_bytes}},
              {{dy, size_t(M) * N * 2}, {ddown ? x : nullptr, nx}, {ddown ? hidden : nullptr, size_t(M) * rank * 4},
               {dx ? down : nullptr, pool * K * 2}, {up, pool * N * 2}, {scales, size_t(adapters) * 4},
               {slots, size_t(M) * 4}, {step, 8}, {dx_add == dx ? nullptr : dx_add, nx}}))
        return WQ_ERR_ARG;
    return wqh::adapters_backward(a, dy, x, hidden, down, up, dx_add, dx, ddown, dup, N, K, workspace,
                                  static_cast<hipStream_t>(stream));
}

extern "C" size_t wq_adapters_backward_workspace_size(int32_t M, int32_t N, int32_t K, int32_t rank,
                                                      int32_t adapters) {
    return sizes_ok(M, N, K, rank, adapters) && rank <= kMaxRank && M > 0
               ? wqh::adapters_backward_workspace(M, N, K, rank, adapters) : 0;
}

extern "C" wq_status wq_dropout(const uint16_t* x, const uint16_t* residual, double p, uint64_t seed, uint64_t offset,
                                const int64_t* step, uint16_t* y, int64_t n, void* stream) {
    wq::Drop d;
    if (n < 0 || n >= (int64_t(1) << 62) || !drop_of(p, seed, offset, step, d)) return WQ_ERR_ARG;
    if (!all_aligned16({x, residual, y})) return WQ_ERR_ARG;
    if (n == 0) return WQ_OK;
    if (!x || !y) return WQ_ERR_ARG;
    const size_t bytes = size_t(n) * 2;
    if (clash({{y, bytes}}, {{x == y ? nullptr : x, bytes}, {residual == y ? nullptr : residual, bytes}, {step, 8}}))
        return WQ_ERR_ARG;
    return wqh::dropout(x, residual, d, y, n, static_cast<hipStream_t>(stream));
}
