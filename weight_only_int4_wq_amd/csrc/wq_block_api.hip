// Entry points of wq_block.h: argument checks, workspace sizes, and the
// choice between the decode-batch and the tiled forward kernels.
#include <initializer_list>

#include "wq_block_common.h"

namespace wqh {
wq_status check_linear_args(const uint16_t* x, const uint32_t* packed, const uint16_t* scales, const uint16_t* y,
                            int M, int N, int K, int bits, int group_size, int* gs_out);
size_t block_bwd_workspace_bytes(int M, int R, int K, int bits, bool has_perm);
wq_status block_bwd(const uint16_t* dy, const uint16_t* preact, int act, bool gated, const uint32_t* packed,
                    const uint16_t* scales, const uint8_t* zeros, const int32_t* perm, const uint16_t* add,
                    uint16_t* dx, uint16_t* dz, float* dbias, int M, int N, int K, int bits, int gs, void* workspace,
                    size_t ws_bytes, hipStream_t s);
}  // namespace wqh

namespace {

bool act_ok(int act) { return act >= WQ_ACT_NONE && act <= WQ_ACT_SILU; }

size_t gather_bytes(int M, int K) { return (size_t(M) * size_t(K) * 2 + 255) & ~size_t(255); }

// The tiled kernels address the rows of one tile with 32-bit byte offsets: 256
// fp16 rows of up to 2^22 channels (or weight rows, 2 I of a gated block).
constexpr int kMaxWidth = 1 << 22;

bool sizes_ok(int M, long long rows, int K) {
    return M >= 0 && M <= (1 << 30) && rows >= 0 && rows <= kMaxWidth && K > 0 && K % 32 == 0 && K <= kMaxWidth;
}

bool query_ok(int M, long long rows, int K, int bits) {
    return sizes_ok(M, rows, K) && M > 0 && rows > 0 && wqh::bits_ok(bits);
}

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

// Bytes of a layer's codes, scales and zero-points.
struct WeightBytes {
    size_t codes, scales, zeros;
    WeightBytes(int rows, int K, int bits, int gs)
        : codes(size_t(rows) * (K / 32) * bits * 4), scales(size_t(rows) * (K / gs) * 2),
          zeros(size_t(rows) * (K / gs)) {}
};

size_t fwd_workspace(int M, int rows, int K, int bits, bool has_perm, bool gated) {
    const size_t part = M <= wqh::kBlockSmallM ? wqh::block_small_part_bytes(M, rows, K, bits, gated)
                                               : wqh::block_fwd_part_bytes(M, rows, K, gated);
    return (has_perm ? gather_bytes(M, K) : 0) + part;
}

wq_status forward(const uint16_t* x, const uint32_t* packed, const uint16_t* scales, const uint8_t* zeros,
                  const int32_t* perm, const uint16_t* bias, const uint16_t* residual, int act, uint16_t* y,
                  uint16_t* preact, int M, int N, int K, int bits, int group_size, bool gated, void* workspace,
                  size_t workspace_bytes, void* stream) {
    if (!sizes_ok(M, gated ? 2LL * N : N, K) || !act_ok(act)) return WQ_ERR_ARG;
    const int rows = gated ? 2 * N : N;
    int gs = 0;
    const wq_status st = wqh::check_linear_args(x, packed, scales, y, M, rows, K, bits, group_size, &gs);
    if (st != WQ_OK) return st;
    for (const void* p : {static_cast<const void*>(perm), static_cast<const void*>(bias),
                          static_cast<const void*>(residual), static_cast<const void*>(preact),
                          static_cast<const void*>(workspace)})
        if (!wqh::aligned16(p)) return WQ_ERR_ARG;
    if (M == 0 || N == 0) return WQ_OK;
    const size_t ny = size_t(M) * N * 2;
    const WeightBytes wb(rows, K, bits, gs);
    if (clash({{y, ny}, {preact, size_t(M) * rows * 2}, {workspace, workspace_bytes}},
              {{x, size_t(M) * K * 2}, {packed, wb.codes}, {scales, wb.scales}, {zeros, wb.zeros},
               {perm, size_t(K) * 4}, {bias, size_t(rows) * 2}, {residual == y ? nullptr : residual, ny}}))
        return WQ_ERR_ARG;
    if (!wqh::block_fwd_fits(M, N, gated)) return WQ_ERR_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    size_t left = workspace ? workspace_bytes : 0;
    if (perm) {
        const size_t need = gather_bytes(M, K);
        if (left < need) return WQ_ERR_ARG;
        const wq_status g = wqh::gather_activations(x, perm, M, K, reinterpret_cast<uint16_t*>(ws), s);
        if (g != WQ_OK) return g;
        x = reinterpret_cast<const uint16_t*>(ws);
        ws += need;
        left -= need;
    }
    const wqh::BlockFwd f{x, packed, scales, zeros, M, rows, K, bits, gs, gated,
                          wq::Epilogue{bias, residual, y, preact, N, act}};
    float* part = reinterpret_cast<float*>(ws);
    if (M <= wqh::kBlockSmallM) {
        // (a K too long for one block's registers without room for partial
        // sums goes to the tiled kernel)
        const wq_status d = wqh::block_small(f, part, left, s);
        if (d != WQ_ERR_UNSUPPORTED) return d;
    }
    return wqh::block_fwd(f, part, left, s);
}

wq_status backward(const uint16_t* dy, const uint16_t* preact, int act, const uint32_t* packed,
                   const uint16_t* scales, const uint8_t* zeros, const int32_t* perm, const uint16_t* dx_add,
                   uint16_t* dx, uint16_t* dz, float* dbias, int M, int N, int K, int bits, int group_size, bool gated,
                   void* workspace, size_t workspace_bytes, void* stream) {
    if (!sizes_ok(M, gated ? 2LL * N : N, K) || !act_ok(act)) return WQ_ERR_ARG;
    if (!wqh::bits_ok(bits)) return WQ_ERR_UNSUPPORTED;
    const int gs = wqh::resolve_group(K, group_size);
    if (!gs) return WQ_ERR_ARG;
    for (const void* p : {static_cast<const void*>(dy), static_cast<const void*>(preact),
                          static_cast<const void*>(packed), static_cast<const void*>(perm),
                          static_cast<const void*>(dx_add), static_cast<const void*>(dx),
                          static_cast<const void*>(dz), static_cast<const void*>(dbias),
                          static_cast<const void*>(workspace)})
        if (!wqh::aligned16(p)) return WQ_ERR_ARG;
    const bool needs_z = gated || act != WQ_ACT_NONE;
    if (M > 0 && !dx) return WQ_ERR_ARG;
    if (M > 0) {
        if (N > 0 && (!dy || !packed || !scales || (needs_z && !preact))) return WQ_ERR_ARG;
        const int rows = gated ? 2 * N : N;
        const size_t nx = size_t(M) * K * 2, nz = size_t(M) * rows * 2;
        const WeightBytes wb(rows, K, bits, gs);
        if (clash({{dx, nx}, {dz, nz}, {dbias, size_t(rows) * 4}, {workspace, workspace_bytes}},
                  {{dy, size_t(M) * N * 2}, {needs_z ? preact : nullptr, nz}, {packed, wb.codes}, {scales, wb.scales},
                   {zeros, wb.zeros}, {perm, size_t(K) * 4}, {dx_add == dx ? nullptr : dx_add, nx}}))
            return WQ_ERR_ARG;
    }
    return wqh::block_bwd(dy, preact, act, gated, packed, scales, zeros, perm, dx_add, dx, dz, dbias, M, N, K, bits, gs,
                          workspace, workspace_bytes, static_cast<hipStream_t>(stream));
}

}  // namespace

extern "C" wq_status wq_linear_act(const uint16_t* x, const uint32_t* packed, const uint16_t* scales,
                                   const uint8_t* zeros, const int32_t* perm, const uint16_t* bias,
                                   const uint16_t* residual, int32_t act, uint16_t* y, uint16_t* preact, int32_t M,
                                   int32_t N, int32_t K, int32_t bits, int32_t group_size, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    return forward(x, packed, scales, zeros, perm, bias, residual, act, y, preact, M, N, K, bits, group_size, false,
                   workspace, workspace_bytes, stream);
}

extern "C" wq_status wq_gated(const uint16_t* x, const uint32_t* packed, const uint16_t* scales, const uint8_t* zeros,
                              const int32_t* perm, const uint16_t* bias, int32_t act, uint16_t* h, uint16_t* preact,
                              int32_t M, int32_t I, int32_t K, int32_t bits, int32_t group_size, void* workspace,
                              size_t workspace_bytes, void* stream) {
    return forward(x, packed, scales, zeros, perm, bias, nullptr, act, h, preact, M, I, K, bits, group_size, true,
                   workspace, workspace_bytes, stream);
}

extern "C" wq_status wq_linear_act_backward(const uint16_t* dy, const uint16_t* preact, int32_t act,
                                            const uint32_t* packed, const uint16_t* scales, const uint8_t* zeros,
                                            const int32_t* perm, const uint16_t* dx_add, uint16_t* dx, uint16_t* dz,
                                            float* dbias, int32_t M, int32_t N, int32_t K, int32_t bits,
                                            int32_t group_size, void* workspace, size_t workspace_bytes,
                                            void* stream) {
    return backward(dy, preact, act, packed, scales, zeros, perm, dx_add, dx, dz, dbias, M, N, K, bits, group_size,
                    false, workspace, workspace_bytes, stream);
}

extern "C" wq_status wq_gated_backward(const uint16_t* dh, const uint16_t* preact, int32_t act,
                                       const uint32_t* packed, const uint16_t* scales, const uint8_t* zeros,
                                       const int32_t* perm, const uint16_t* dx_add, uint16_t* dx, uint16_t* dz,
                                       float* dbias, int32_t M, int32_t I, int32_t K, int32_t bits,
                                       int32_t group_size, void* workspace, size_t workspace_bytes, void* stream) {
    return backward(dh, preact, act, packed, scales, zeros, perm, dx_add, dx, dz, dbias, M, I, K, bits, group_size,
                    true, workspace, workspace_bytes, stream);
}

extern "C" size_t wq_linear_act_workspace_size(int32_t M, int32_t N, int32_t K, int32_t bits, int32_t has_perm) {
    return query_ok(M, N, K, bits) ? fwd_workspace(M, N, K, bits, has_perm != 0, false) : 0;
}

extern "C" size_t wq_gated_workspace_size(int32_t M, int32_t I, int32_t K, int32_t bits, int32_t has_perm) {
    return query_ok(M, 2LL * I, K, bits) ? fwd_workspace(M, 2 * I, K, bits, has_perm != 0, true) : 0;
}

extern "C" size_t wq_linear_act_backward_workspace_size(int32_t M, int32_t N, int32_t K, int32_t bits,
                                                        int32_t has_perm) {
    return query_ok(M, N, K, bits) ? wqh::block_bwd_workspace_bytes(M, N, K, bits, has_perm != 0) : 0;
}

extern "C" size_t wq_gated_backward_workspace_size(int32_t M, int32_t I, int32_t K, int32_t bits, int32_t has_perm) {
    return query_ok(M, 2LL * I, K, bits) ? wqh::block_bwd_workspace_bytes(M, 2 * I, K, bits, has_perm != 0) : 0;
}
