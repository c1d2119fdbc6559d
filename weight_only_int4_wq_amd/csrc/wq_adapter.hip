// Low-rank adapters beside a quantized layer, forward and backward
// (wq_adapter.h), on the matrix cores.
//
// Both passes are the same two products, each along its long side, and the
// backward pass has a third:
//   shrink:  h[m][r]     = sum over c of src[m][c] w[a][r][c]      (x with down, dy with up)
//   expand:  out[m][c]   = add[m][c] + s sum over r of h[m][r] w[a][r][c]   (h with up, dh with down)
//   outer:   dw[a][r][c] = s sum over a's rows m of h[m][r] src[m][c]       (dh with x, hidden with dy)
// Every adapter array is [rank][C] with C contiguous, so that two kernels
// serve both directions.
//
// Rows come with any adapter in any order.  A block looks at a window of 64
// rows, and for each adapter that occurs in it gathers that adapter's rows
// into 16-row matrix fragments: runs of one adapter fill them, and a decode
// batch reads each adapter once per window.  Neither sorting nor a plan is
// needed, and no row sees another adapter's weights, whose infinities would
// turn a masked product into NaN.
#include "wq_adapter_common.h"

namespace {

using wq::Drop;
using wq::f4;
using wq::h8;
using wq::u4;

constexpr int kWindow = 64;   // rows a block looks at: a wavefront's lanes
constexpr int kChunk = 128;   // columns of src that a wavefront takes at a time
constexpr int kCols = 128;    // columns of out and dw of a wavefront: 16 lanes of 8

// Eight fp16 values at p, which need not be aligned to more than one of them
// (odd row lengths): the hardware takes 16-byte accesses at any address.
__device__ __forceinline__ u4 load8(const uint16_t* p) {
    u4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
// The first n of them (n <= 0: none), zeros behind.
__device__ __forceinline__ u4 load8_part(const uint16_t* p, int n) {
    if (n >= 8) return load8(p);
    u4 v{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) v[i >> 1] |= uint32_t(p[i]) << (16 * (i & 1));
    return v;
}
__device__ __forceinline__ void store8_part(uint16_t* p, u4 v, int n) {
    if (n >= 8) {
        __builtin_memcpy(p, &v, 16);
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) p[i] = uint16_t(v[i >> 1] >> (16 * (i & 1)));
}

__device__ __forceinline__ f4 mfma(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// Rows 8 g + i of a fragment's k dimension as 8 loads of 8 neighbouring
// columns, to the fragments of those columns: fragment j holds column j of the
// lane's eight (matrix column 8 (l % 16) + j), so a lane ends up with eight
// neighbouring columns of the result.
__device__ __forceinline__ void transpose8(const u4 (&row)[8], u4 (&frag)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            frag[j][q] = __builtin_amdgcn_perm(row[2 * q + 1][j >> 1], row[2 * q][j >> 1],
                                               j & 1 ? 0x07060302u : 0x05040100u);
}

typedef uint16_t us2 __attribute__((ext_vector_type(2)));

// All ones in the halves of w that are at least t (t > 0).
__device__ __forceinline__ uint32_t keep_mask(uint32_t w, us2 below) {
    const us2 over = __builtin_elementwise_sub_sat(__builtin_bit_cast(us2, w), below);  // w - (t - 1), 0 at least
    const us2 one = __builtin_elementwise_min(over, us2{1, 1});
    return __builtin_bit_cast(uint32_t, us2{0, 0} - one);
}
// Eight values with the dropped ones zeroed; n: the eight's number.
__device__ __forceinline__ u4 drop8(u4 v, uint64_t n, const Drop& d, uint64_t stream) {
    const u4 w = wq::philox(n, stream, d.key0, d.key1);
    const us2 below{uint16_t(d.t - 1), uint16_t(d.t - 1)};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] &= keep_mask(w[i], below);
    return v;
}

// Lane l's row of a window: its slot, -1 for one without an adapter.
__device__ __forceinline__ int slot_of(const int32_t* slots, int64_t m, int M, int L) {
    if (m >= M) return -1;
    const int s = slots ? slots[m] : 0;
    return unsigned(s) < unsigned(L) ? s : -1;
}
// The lanes in `mask` first, in order, then the others: lane i gets the i-th's number.
__device__ __forceinline__ int compact(uint64_t mask) {
    const int lane = threadIdx.x & 63;
    const int below = __builtin_amdgcn_mbcnt_hi(uint32_t(mask >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(mask), 0));
    const int to = mask >> lane & 1 ? below : __builtin_popcountll(mask) + lane - below;
    return __builtin_amdgcn_ds_permute(to * 4, lane);
}

// Calls work(adapter, rows, order) for the window's adapters z, z + Z, ... in
// order of appearance; order: the adapter's rows first.
template <class Work>
__device__ __forceinline__ void each_adapter(int slot, int z, int Z, const Work& work) {
    uint64_t todo = __ballot(slot >= 0);
    for (int n = 0; todo; ++n) {
        const int a = __builtin_amdgcn_readlane(slot, __builtin_ctzll(todo));
        const uint64_t mine = __ballot(slot == a);
        todo &= ~mine;
        if (n % Z == z) work(a, __builtin_popcountll(mine), compact(mine));
    }
}

// 2^k that brings a largest magnitude `most` (finite) into [2^top, 2^(top + 1)),
// within fp32's normal numbers, and its inverse.
__device__ __forceinline__ float to_range(float most, int top, float& inverse) {
    const int e = int(__builtin_bit_cast(uint32_t, most) >> 23);
    const int k = min(top + 127 - e, 126);
    inverse = __builtin_bit_cast(float, uint32_t(127 - k) << 23);
    return __builtin_bit_cast(float, uint32_t(127 + k) << 23);
}
__device__ __forceinline__ float finite_magnitude(float v) {
    const float a = __builtin_fabsf(v);
    return a <= 3.402823466e38f ? a : 0.f;
}
// v as a sum of two fp16 numbers (an infinity: itself and zero).
__device__ __forceinline__ void split_h(float v, uint16_t& hi, uint16_t& lo) {
    const _Float16 h = (_Float16)v;
    const float f = float(h);
    hi = __builtin_bit_cast(uint16_t, h);
    lo = wq::f2h(v == f ? 0.f : v - f);
}

// --------------------------------------------------------------- shrink ----

struct Shrink {
    const uint16_t* src;   // [M][C]
    const uint16_t* w;     // [L][R][C]
    const int32_t* slots;
    float* part;           // [splits][M][RP], columns past R zero
    Drop drop;
    int M, R, L, C;
    int splits, cps;       // ranges of columns, in chunks of 128
    int Z, rchunks;        // blocks that share a window's adapters; 64-wide ranges of the rank
    // rows by adapter, for the gradients (null: not wanted)
    int32_t* start;        // [L + 1]
    int32_t* list;         // [M]
    int64_t blocks;        // of the product; those behind them make the lists
};

// Lists of rows by adapter: a wavefront per adapter counts the rows of lower
// ones (its start) and writes its own in order.  2 M / 64 loads a wavefront, next to
// the product's blocks.
__device__ __forceinline__ void list_rows(const Shrink& p, int64_t a) {
    const int lane = threadIdx.x & 63;
    if (a >= p.L) return;
    constexpr int U = 8;
    int less = 0, mine = 0;
    for (int64_t m = 0; m < p.M; m += 64 * U) {
        int s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = slot_of(p.slots, m + 64 * u + lane, p.M, p.L);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            less += s[u] >= 0 && s[u] < a;
            mine += s[u] == a;
        }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        less += __shfl_xor(less, o);
        mine += __shfl_xor(mine, o);
    }
    if (lane == 0) {
        p.start[a] = less;
        if (a == p.L - 1) p.start[p.L] = less + mine;
    }
    if (!mine) return;
    for (int64_t m = 0; m < p.M; m += 64 * U) {
        int s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = slot_of(p.slots, m + 64 * u + lane, p.M, p.L);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint64_t mask = __ballot(s[u] == a);
            const int at = less + __builtin_amdgcn_mbcnt_hi(uint32_t(mask >> 32),
                                                            __builtin_amdgcn_mbcnt_lo(uint32_t(mask), 0));
            if (s[u] == a) p.list[at] = int(m + 64 * u + lane);
            less += __builtin_popcountll(mask);
        }
    }
}

// One adapter's rows of a window against 16 NRT of its rank's rows, over the
// block's range of columns; the four wavefronts take its chunks in turn.
template <int MT, int NRT, bool DROP>
__device__ __forceinline__ void shrink_rows(const Shrink& p, int64_t m0, int a, int cnt, int order, int r0, int split, f4* sum) {
    // columns a wavefront loads at a time: 32 to a matrix step
    constexpr int STEPS = MT + NRT > 5 ? 2 : 4, COLS = 32 * STEPS;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, g = lane >> 4;
    f4 acc[MT][NRT];
    const uint16_t* xr[MT];
    uint64_t eight[MT];
    bool on[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t m = m0 + __shfl(order, 16 * t + c16);
        on[t] = 16 * t + c16 < cnt;
        xr[t] = p.src + m * p.C + 8 * g;
        eight[t] = uint64_t(m) * (p.C / 8) + g;
#pragma unroll
        for (int n = 0; n < NRT; ++n) acc[t][n] = f4{0.f, 0.f, 0.f, 0.f};
    }
    const uint16_t* wr[NRT];   // (rows past the rank repeat the last one: their columns of h become zeros)
#pragma unroll
    for (int n = 0; n < NRT; ++n) wr[n] = p.w + (int64_t(a) * p.R + min(r0 + 16 * n + c16, p.R - 1)) * p.C + 8 * g;
    const uint64_t stream = DROP ? wq::drop_stream(p.drop) : 0;

    u4 x[2][MT][STEPS], w[2][NRT][STEPS];
    auto load = [&](int64_t c0, u4 (&xs)[MT][STEPS], u4 (&ws)[NRT][STEPS]) {
        if (c0 + COLS <= p.C) {
#pragma unroll
            for (int n = 0; n < NRT; ++n)
#pragma unroll
                for (int i = 0; i < STEPS; ++i) ws[n][i] = load8(wr[n] + c0 + 32 * i);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    xs[t][i] = u4{0, 0, 0, 0};
                    if (on[t]) xs[t][i] = load8(xr[t] + c0 + 32 * i);
                }
        } else {
            const int left = int(p.C - c0) - 8 * g;
#pragma unroll
            for (int n = 0; n < NRT; ++n)
#pragma unroll
                for (int i = 0; i < STEPS; ++i) ws[n][i] = load8_part(wr[n] + c0 + 32 * i, left - 32 * i);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < STEPS; ++i)
                    xs[t][i] = load8_part(xr[t] + c0 + 32 * i, on[t] ? left - 32 * i : 0);
        }
    };
    auto multiply = [&](int64_t c0, u4 (&xs)[MT][STEPS], u4 (&ws)[NRT][STEPS]) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if constexpr (DROP) xs[t][i] = drop8(xs[t][i], eight[t] + uint64_t(c0 / 8 + 4 * i), p.drop, stream);
#pragma unroll
                for (int n = 0; n < NRT; ++n) acc[t][n] = mfma(xs[t][i], ws[n][i], acc[t][n]);
            }
    };
    const int64_t end = min(int64_t(split + 1) * p.cps * kChunk, int64_t(p.C));
    int64_t c0 = int64_t(split) * p.cps * kChunk + wave * COLS;
    if (c0 < end) load(c0, x[0], w[0]);
    for (; c0 < end; c0 += 8 * COLS) {
        const int64_t c1 = c0 + 4 * COLS, c2 = c1 + 4 * COLS;
        if (c1 < end) load(c1, x[1], w[1]);
        multiply(c0, x[0], w[0]);
        if (c2 < end) load(c2, x[0], w[0]);
        if (c1 < end) multiply(c1, x[1], w[1]);
    }

    // the four wavefronts' sums, in order
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NRT; ++n) sum[((t * NRT + n) * 4 + wave) * 64 + lane] = acc[t][n];
    __syncthreads();
    const int RP = NRT * 16 * p.rchunks;
    for (int e = wave; e < MT * NRT; e += 4) {
        const int t = e / NRT, n = e % NRT, r = r0 + 16 * n + c16;
        f4 v = sum[e * 256 + lane];
#pragma unroll
        for (int i = 1; i < 4; ++i) v += sum[e * 256 + 64 * i + lane];
        const float f = r < p.R ? DROP ? p.drop.keep : 1.f : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * t + 4 * g + i;
            const int64_t m = m0 + __shfl(order, row);
            if (row < cnt) p.part[(int64_t(split) * p.M + m) * RP + r] = r < p.R ? v[i] * f : 0.f;
        }
    }
    __syncthreads();
}

// Blocks: for a window, its ranges of columns (neighbouring blocks: the XCDs
// take them in turn, so that each holds its own range of every adapter in L2),
// the rank's 64s, and Z shares of its adapters.
template <int NRT, bool DROP>
__global__ __launch_bounds__(256) void shrink_kernel(const Shrink p, int64_t first) {
    __shared__ f4 sum[4 * NRT * 256];
    int64_t b = first + blockIdx.x;
    if (b >= p.blocks) {
        list_rows(p, (b - p.blocks) * 4 + (threadIdx.x >> 6));
        return;
    }
    const int split = int(b % p.splits);
    b /= p.splits;
    const int r0 = int(b % p.rchunks) * 64;
    b /= p.rchunks;
    const int z = int(b % p.Z);
    const int64_t m0 = b / p.Z * kWindow;
    const int slot = slot_of(p.slots, m0 + (threadIdx.x & 63), p.M, p.L);
    each_adapter(slot, z, p.Z, [&](int a, int cnt, int order) {
        if (cnt <= 16)
            shrink_rows<1, NRT, DROP>(p, m0, a, cnt, order, r0, split, sum);
        else if (cnt <= 32)
            shrink_rows<2, NRT, DROP>(p, m0, a, cnt, order, r0, split, sum);
        else
            shrink_rows<4, NRT, DROP>(p, m0, a, cnt, order, r0, split, sum);
    });
}

// --------------------------------------------------------------- expand ----

struct Expand {
    const float* part;     // [splits][M][RP]
    const uint16_t* w;     // [L][R][C]
    const float* scales;
    const int32_t* slots;
    const uint16_t* add;   // [M][C], nullable, may be out
    uint16_t* out;         // [M][C]
    float* sum;            // h [M][R], nullable
    Drop drop;
    int M, R, L, C, splits;
    int Z, span, cblocks;  // a block's columns: span * 512
};

template <int RP>
struct ExpandTile {
    // A fragment of 32: the first fp16 parts in its lower half, the second
    // parts in its upper half where the rank fits 16, else one after the other.
    static constexpr bool BOTH = RP == 16;
    static constexpr int KB = BOTH ? 1 : RP / 32;   // 32-row pieces of w
    static constexpr int STRIDE = 2 * RP + 8;       // halves to a row in LDS, 16-byte aligned
};

template <int RP, bool DROP>
__global__ __launch_bounds__(256) void expand_kernel(const Expand p, int64_t total, int64_t first) {
    typedef ExpandTile<RP> T;
    __shared__ __attribute__((aligned(16))) uint16_t parts[kWindow * T::STRIDE];
    __shared__ __attribute__((aligned(16))) float back[kWindow];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, g = lane >> 4;
    // contiguous tiles to an XCD: a window's column blocks share its h
    int64_t b = first + blockIdx.x;
    {
        const int64_t q = total / 8, r = total % 8, x = b % 8, k = b / 8;
        b = x < r ? x * (q + 1) + k : r * (q + 1) + (x - r) * q + k;
    }
    const int cb = int(b % p.cblocks);
    b /= p.cblocks;
    const int z = int(b % p.Z);
    const int64_t m0 = b / p.Z * kWindow;
    const int slot = slot_of(p.slots, m0 + lane, p.M, p.L);
    const int64_t col0 = (int64_t(cb) * p.span * 4 + wave) * kCols + 8 * c16;   // the lane's first column
    const uint64_t stream = DROP ? wq::drop_stream(p.drop) : 0;

    each_adapter(slot, z, p.Z, [&](int a, int cnt, int order) {
        // h of the adapter's rows, four threads to a row: summed over the
        // ranges, scaled into fp16's range row by row and split in two
        {
            const int row = threadIdx.x >> 2, q = threadIdx.x & 3;
            const int64_t m = m0 + __shfl(order, row);
            f4 v[RP / 16];
#pragma unroll
            for (int i = 0; i < RP / 16; ++i) v[i] = f4{0.f, 0.f, 0.f, 0.f};
            if (row < cnt)
                for (int s = 0; s < p.splits; ++s) {
                    const float* h = p.part + (int64_t(s) * p.M + m) * RP + q * (RP / 4);
#pragma unroll
                    for (int i = 0; i < RP / 16; ++i) v[i] += *reinterpret_cast<const f4*>(h + 4 * i);
                }
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < RP / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) most = __builtin_fmaxf(most, finite_magnitude(v[i][j]));
            most = __builtin_fmaxf(most, __shfl_xor(most, 1));
            most = __builtin_fmaxf(most, __shfl_xor(most, 2));
            float inverse;
            const float scale = to_range(most, 13, inverse);
            if (q == 0) back[row] = inverse;
            uint16_t* to = parts + row * T::STRIDE + q * (RP / 4);
#pragma unroll
            for (int i = 0; i < RP / 16; ++i) {
                uint16_t hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) split_h(v[i][j] * scale, hi[j], lo[j]);
                __builtin_memcpy(__builtin_assume_aligned(to + 4 * i, 8), hi, 8);
                __builtin_memcpy(__builtin_assume_aligned(to + RP + 4 * i, 8), lo, 8);
            }
            if (p.sum && cb == 0 && row < cnt)
#pragma unroll
                for (int i = 0; i < RP / 16; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = q * (RP / 4) + 4 * i + j;
                        if (r < p.R) p.sum[m * p.R + r] = v[i][j];
                    }
        }
        __syncthreads();
        const float s = p.scales[a] * (DROP ? p.drop.keep : 1.f);
        const int tiles = (cnt + 15) / 16;
        for (int ct = 0; ct < p.span; ++ct) {
            const int64_t c = col0 + int64_t(ct) * 4 * kCols;
            if (!p.out || c - 8 * c16 >= p.C) break;
            const int left = int(p.C - c);
            u4 w[T::KB][8];
#pragma unroll
            for (int k = 0; k < T::KB; ++k) {
                u4 raw[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // (rows past the rank are zeros, not the next adapter's)
                    const int r = T::BOTH ? 8 * (g & 1) + i : 32 * k + 8 * g + i;
                    raw[i] = load8_part(p.w + (int64_t(a) * p.R + r) * p.C + c, r < p.R ? left : 0);
                }
                transpose8(raw, w[k]);
            }
            for (int t = 0; t < tiles; ++t) {
                int64_t m[4];
                u4 old[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * t + 4 * g + i;
                    m[i] = m0 + __shfl(order, row);
                    old[i] = u4{0, 0, 0, 0};
                    if (p.add && row < cnt) old[i] = load8_part(p.add + m[i] * p.C + c, left);
                }
                f4 acc[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = f4{0.f, 0.f, 0.f, 0.f};
                const uint16_t* h = parts + (16 * t + c16) * T::STRIDE + 8 * g;
#pragma unroll
                for (int k = 0; k < T::KB; ++k) {
                    const u4 hi = *reinterpret_cast<const u4*>(h + 32 * k);
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[j] = mfma(hi, w[k][j], acc[j]);
                    if constexpr (!T::BOTH) {
                        const u4 lo = *reinterpret_cast<const u4*>(h + RP + 32 * k);
#pragma unroll
                        for (int j = 0; j < 8; ++j) acc[j] = mfma(lo, w[k][j], acc[j]);
                    }
                }
                const f4 inverse = *reinterpret_cast<const f4*>(back + 16 * t + 4 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (16 * t + 4 * g + i >= cnt) continue;
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = acc[j][i] * inverse[i] * s;
                    if constexpr (DROP) {
                        const u4 d = wq::philox((uint64_t(m[i]) * p.C + c) >> 3, stream, p.drop.key0, p.drop.key1);
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] = wq::kept(d, j, p.drop.t) ? f[j] : 0.f;
                    }
                    uint16_t o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float before = wq::h2f(uint16_t(old[i][j >> 1] >> (16 * (j & 1))));
                        o[j] = wq::f2h(p.add ? before + f[j] : f[j]);
                    }
                    u4 v;
                    __builtin_memcpy(&v, o, 16);
                    store8_part(p.out + m[i] * p.C + c, v, left);
                }
            }
        }
        __syncthreads();
    });

    // rows without an adapter
    const uint64_t none = z == 0 ? __ballot(slot < 0 && m0 + lane < p.M) : 0;
    if (!none) return;
    const int cnt = __builtin_popcountll(none), order = compact(none);
    if (p.out && p.out != p.add)
        for (int ct = 0; ct < p.span; ++ct) {
            const int64_t c = col0 + int64_t(ct) * 4 * kCols;
            if (c - 8 * c16 >= p.C) break;
            const int left = int(p.C - c);
            for (int row = 0; row < cnt; row += 4) {
                const int64_t m = m0 + __shfl(order, row + g);
                if (row + g >= cnt) continue;
                store8_part(p.out + m * p.C + c, p.add ? load8_part(p.add + m * p.C + c, left) : u4{0, 0, 0, 0}, left);
            }
        }
    if (p.sum && cb == 0)
        for (int i0 = 0; i0 < cnt * p.R; i0 += 256) {
            const int i = i0 + threadIdx.x;
            const int64_t m = m0 + __shfl(order, (i / p.R) & 63);
            if (i < cnt * p.R) p.sum[m * p.R + i % p.R] = 0.f;
        }
}

// ---------------------------------------------------------------- outer ----

// One gradient: dw [L][R][C] of h [M][R] and src [M][C].
struct OuterJob {
    const float* h;
    const uint16_t* src;
    float* dw;
    float* part;           // [splits][L][R][C] where splits > 1
    Drop drop;
    int C, tiles;  // tiles of 128 columns
};
struct Outer {
    OuterJob job[2];
    const float* scales;
    const int32_t* start;  // [L + 1], null: adapter 0 takes every row
    const int32_t* list;
    int M, R, L, splits, rchunks;
    int64_t blocks0;       // blocks of job 0
};

// Rows of one adapter, 32 to a matrix step, against 128 columns: a block's
// wavefronts take steps in turn.  h is brought into fp16's range for each of its
// columns r, by a power of two that follows the largest magnitude so far, with
// room for it to grow 2^5 times before the sums are rescaled.
template <int NRT>
__global__ __launch_bounds__(256) void outer_kernel(const Outer p, int64_t first) {
    __shared__ f4 sums[2 * NRT * 8 * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, g = lane >> 4;
    int64_t b = first + blockIdx.x;
    const bool second = b >= p.blocks0;
    if (second) b -= p.blocks0;
    const OuterJob& j = p.job[second];
    const int tile = int(b % j.tiles);
    b /= j.tiles;
    const int split = int(b % p.splits);
    b /= p.splits;
    const int r0 = int(b % p.rchunks) * 64;
    const int a = int(b / p.rchunks);
    const int at = p.start ? p.start[a] : 0, cnt = p.start ? p.start[a + 1] - at : a == 0 ? p.M : 0;
    const int64_t c = int64_t(tile) * kCols + 8 * c16;
    const int left = int(j.C - c);
    const bool drop = j.drop.t != 0;
    const uint64_t stream = drop ? wq::drop_stream(j.drop) : 0;
    const int steps = (cnt + 31) / 32;
    const int end = int(int64_t(split + 1) * steps / p.splits);
    const int rl = r0 + NRT * c16;       // the lane's first r; fragment t holds r0 + NRT (l % 16) + t
    f4 acc[NRT][8];
    float mul[NRT];
#pragma unroll
    for (int t = 0; t < NRT; ++t) {
        mul[t] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[t][i] = f4{0.f, 0.f, 0.f, 0.f};
    }

    for (int st = int(int64_t(split) * steps / p.splits) + wave; st < end; st += 4) {
        const int i0 = st * 32 + 8 * g;
        u4 x[8];
        float h[8][NRT];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool on = i0 + i < cnt;
            const int64_t m = !on ? 0 : p.list ? p.list[at + i0 + i] : i0 + i;
            x[i] = load8_part(j.src + m * j.C + c, on ? left : 0);
            const float* hp = j.h + m * p.R + rl;
#pragma unroll
            for (int t = 0; t < NRT; ++t) h[i][t] = 0.f;
            if (on && rl + NRT <= p.R) {
                __builtin_memcpy(h[i], hp, 4 * NRT);
            } else if (on) {
#pragma unroll
                for (int t = 0; t < NRT; ++t)
                    if (rl + t < p.R) h[i][t] = hp[t];
            }
            if (drop) x[i] = drop8(x[i], (uint64_t(m) * j.C + c) >> 3, j.drop, stream);
        }
        float most[NRT];
        bool grow = false;
#pragma unroll
        for (int t = 0; t < NRT; ++t) {
            most[t] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) most[t] = __builtin_fmaxf(most[t], finite_magnitude(h[i][t]));
            most[t] = __builtin_fmaxf(most[t], __shfl_xor(most[t], 16));
            most[t] = __builtin_fmaxf(most[t], __shfl_xor(most[t], 32));
            grow |= most[t] * mul[t] >= 32768.f || (mul[t] == 0.f && most[t] > 0.f);
        }
        if (__ballot(grow)) {
#pragma unroll
            for (int t = 0; t < NRT; ++t) {
                float ratio = 1.f;
                if (most[t] * mul[t] >= 32768.f || (mul[t] == 0.f && most[t] > 0.f)) {
                    float inverse;
                    const float next = to_range(most[t], 9, inverse);
                    ratio = mul[t] == 0.f ? 1.f : next / mul[t];
                    mul[t] = next;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = __shfl(ratio, 4 * g + i);
#pragma unroll
                    for (int k = 0; k < 8; ++k) acc[t][k][i] *= f;
                }
            }
        }
        u4 w[8];
        transpose8(x, w);
#pragma unroll
        for (int t = 0; t < NRT; ++t) {
            const float scale = mul[t] == 0.f ? 1.f : mul[t];
            uint16_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) split_h(h[i][t] * scale, hi[i], lo[i]);
            u4 vh, vl;
            __builtin_memcpy(&vh, hi, 16);
            __builtin_memcpy(&vl, lo, 16);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[t][k] = mfma(vh, w[k], acc[t][k]);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[t][k] = mfma(vl, w[k], acc[t][k]);
        }
    }

    // back from the powers of two, then (0 + 2) + (1 + 3)
    const float s = (drop ? j.drop.keep : 1.f) * (cnt ? p.scales[a] : 0.f);
#pragma unroll
    for (int t = 0; t < NRT; ++t) {
        const float inverse = mul[t] == 0.f ? 1.f : 1.f / mul[t];   // (a power of two: exact)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = __shfl(inverse, 4 * g + i);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[t][k][i] *= f;
        }
    }
    auto give = [&](f4* to) {
#pragma unroll
        for (int t = 0; t < NRT; ++t)
#pragma unroll
            for (int k = 0; k < 8; ++k) to[(t * 8 + k) * 64 + lane] = acc[t][k];
    };
    auto take = [&](const f4* from) {
#pragma unroll
        for (int t = 0; t < NRT; ++t)
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[t][k] += from[(t * 8 + k) * 64 + lane];
    };
    f4* const half = sums + NRT * 8 * 64;
    if (wave >= 2) give(wave == 2 ? sums : half);
    __syncthreads();
    if (wave < 2) take(wave == 0 ? sums : half);
    __syncthreads();
    if (wave == 1) give(sums);
    __syncthreads();
    if (wave != 0) return;
    take(sums);

    float* to = p.splits > 1 ? j.part + int64_t(split) * p.L * p.R * j.C : j.dw;
#pragma unroll
    for (int t = 0; t < NRT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + NRT * (4 * g + i) + t;
            if (r >= p.R) continue;
            float* row = to + (int64_t(a) * p.R + r) * j.C + c;
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = acc[t][k][i] * s;
            if (left >= 8) {
                __builtin_memcpy(row, v, 32);
            } else {
#pragma unroll
                for (int k = 0; k < 7; ++k)
                    if (k < left) row[k] = v[k];
            }
        }
}

// dw = the sum over the ranges of rows, in order; four values to a thread.
__global__ __launch_bounds__(256) void outer_sum_kernel(const Outer p, int64_t n0, int64_t first) {
    int64_t q = (first + int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
    const bool second = q >= n0;
    if (second) q -= n0;
    const OuterJob& j = p.job[second];
    const int64_t size = int64_t(p.L) * p.R * j.C;
    if (q >= size) return;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    const int k = int(min(size - q, int64_t(4)));
    for (int s = 0; s < p.splits; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < k) v[i] += j.part[s * size + q + i];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < k) j.dw[q + i] = v[i];
}

// -------------------------------------------------------------- launches ----

constexpr Drop kNoDrop{0, 1.f, 0, 0, 0, nullptr};

int div_up(int64_t a, int64_t b) { return int((a + b - 1) / b); }
size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

int padded_rank(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128; }

template <class Launch>
wq_status pieces(int64_t blocks, const Launch& launch) {
    for (int64_t first = 0; first < blocks; first += wqh::kMaxBlocks) {
        launch(unsigned(std::min<int64_t>(blocks - first, wqh::kMaxBlocks)), first);
        const wq_status st = wqh::launch_status();
        if (st != WQ_OK) return st;
    }
    return WQ_OK;
}

// Ranges of the long side of a shrink, and the blocks that share a window.
struct ShrinkPlan {
    int splits, cps, Z;
    ShrinkPlan(int M, int R, int L, int C) {
        const int chunks = div_up(C, kChunk), rchunks = padded_rank(R) > 64 ? 2 : 1;
        const int64_t base = int64_t(div_up(M, kWindow)) * rchunks;
        const int want = int(std::min<int64_t>(std::max<int64_t>(768 / base, 1), 32));
        cps = div_up(chunks, std::min(want, div_up(chunks, 4)));
        splits = div_up(chunks, cps);
        Z = int(std::max<int64_t>(1, std::min<int64_t>(std::min(std::min(L, M), kWindow), 768 / (base * splits))));
    }
    size_t bytes(int M, int R) const { return round256(size_t(splits) * M * padded_rank(R) * 4); }
};

wq_status shrink(const wqh::Adapters& a, const uint16_t* src, const uint16_t* w, const Drop& d, float* part, int C,
                 int32_t* start, int32_t* list, hipStream_t s) {
    const ShrinkPlan plan(a.M, a.R, a.L, C);
    const int RP = padded_rank(a.R);
    Shrink p{src, w, a.slots, part, d, a.M, a.R, a.L, C, plan.splits, plan.cps, plan.Z, RP > 64 ? 2 : 1, start, list, 0};
    p.blocks = int64_t(div_up(a.M, kWindow)) * p.splits * p.Z * p.rchunks;
    const int64_t all = p.blocks + (start ? div_up(a.L, 4) : 0);
    return pieces(all, [&](unsigned blocks, int64_t first) {
        auto go = [&](auto n) {
            if (d.t)
                shrink_kernel<decltype(n)::value, true><<<blocks, 256, 0, s>>>(p, first);
            else
                shrink_kernel<decltype(n)::value, false><<<blocks, 256, 0, s>>>(p, first);
        };
        if (RP == 16)
            go(std::integral_constant<int, 1>{});
        else if (RP == 32)
            go(std::integral_constant<int, 2>{});
        else
            go(std::integral_constant<int, 4>{});
    });
}

wq_status expand(const wqh::Adapters& a, const float* part, int splits, const uint16_t* w, const Drop& d,
                 const uint16_t* add, uint16_t* out, float* sum, int C, hipStream_t s) {
    const int64_t windows = div_up(a.M, kWindow);
    const int wide = out ? div_up(C, 4 * kCols) : 1;   // blocks of 512 columns
    Expand p{part, w, a.scales, a.slots, add, out, sum, d, a.M, a.R, a.L, C, splits, 1, 1, 1};
    p.span = int(std::max<int64_t>(1, std::min<int64_t>(std::min(wide, 8), windows * wide / 768)));
    p.cblocks = div_up(wide, p.span);
    p.Z = int(std::max<int64_t>(1, std::min<int64_t>(std::min(std::min(a.L, a.M), kWindow), 512 / (windows * p.cblocks))));
    const int64_t all = windows * p.cblocks * p.Z;
    return pieces(all, [&](unsigned blocks, int64_t first) {
        auto go = [&](auto n) {
            if (d.t)
                expand_kernel<decltype(n)::value, true><<<blocks, 256, 0, s>>>(p, all, first);
            else
                expand_kernel<decltype(n)::value, false><<<blocks, 256, 0, s>>>(p, all, first);
        };
        switch (padded_rank(a.R)) {
            case 16: go(std::integral_constant<int, 16>{}); break;
            case 32: go(std::integral_constant<int, 32>{}); break;
            case 64: go(std::integral_constant<int, 64>{}); break;
            default: go(std::integral_constant<int, 128>{});
        }
    });
}

// Ranges of rows of the gradients.
int outer_splits(int M, int R, int L, int K, int N) {
    const int64_t blocks = int64_t(L) * (padded_rank(R) > 64 ? 2 : 1) * (div_up(K, kCols) + div_up(N, kCols));
    return int(std::max<int64_t>(1, std::min<int64_t>(std::min(div_up(M, 128), 32), 768 / blocks)));
}

wq_status outer(const wqh::Adapters& a, Outer& p, hipStream_t s) {
    const int RP = padded_rank(a.R);
    p.rchunks = RP > 64 ? 2 : 1;
    const int64_t per = int64_t(a.L) * p.rchunks * p.splits;
    for (OuterJob& j : p.job) j.tiles = div_up(j.C, kCols);
    p.blocks0 = per * p.job[0].tiles;
    wq_status st = pieces(p.blocks0 + per * p.job[1].tiles, [&](unsigned blocks, int64_t first) {
        if (RP == 16)
            outer_kernel<1><<<blocks, 256, 0, s>>>(p, first);
        else if (RP == 32)
            outer_kernel<2><<<blocks, 256, 0, s>>>(p, first);
        else
            outer_kernel<4><<<blocks, 256, 0, s>>>(p, first);
    });
    if (st != WQ_OK || p.splits == 1) return st;
    const int64_t n0 = (int64_t(a.L) * a.R * p.job[0].C + 3) / 4 * 4, n1 = int64_t(a.L) * a.R * p.job[1].C;
    return pieces((n0 + n1 + 1023) / 1024, [&](unsigned blocks, int64_t first) {
        outer_sum_kernel<<<blocks, 256, 0, s>>>(p, n0, first * 256);
    });
}

// The backward pass's workspace.
struct BackwardRoom {
    size_t part, dh, start, list, outer0, outer1, bytes;
    int splits;
    BackwardRoom(int M, int N, int K, int R, int L) {
        splits = outer_splits(M, R, L, K, N);
        const size_t grads = splits > 1 ? size_t(splits) * L * R * 4 : 0;
        size_t at = 0;
        auto take = [&](size_t n) {
            const size_t was = at;
            at += round256(n);
            return was;
        };
        part = take(ShrinkPlan(M, R, L, N).bytes(M, R));
        dh = take(size_t(M) * R * 4);
        start = take((size_t(L) + 1) * 4);
        list = take(size_t(M) * 4);
        outer0 = take(grads * K);
        outer1 = take(grads * N);
        bytes = at;
    }
};

}  // namespace

namespace wqh {

size_t adapters_workspace(int M, int, int K, int R, int L) { return ShrinkPlan(M, R, L, K).bytes(M, R); }

wq_status adapters_forward(const Adapters& a, const uint16_t* x, const uint16_t* down, const uint16_t* up,
                           const uint16_t* base, uint16_t* y, float* hidden, int N, int K, void* ws, hipStream_t s) {
    float* part = static_cast<float*>(ws);
    const wq_status st = shrink(a, x, down, a.drop, part, K, nullptr, nullptr, s);
    return st != WQ_OK ? st
                       : expand(a, part, ShrinkPlan(a.M, a.R, a.L, K).splits, up, kNoDrop, base, y, hidden, N, s);
}

size_t adapters_backward_workspace(int M, int N, int K, int R, int L) { return BackwardRoom(M, N, K, R, L).bytes; }

wq_status adapters_backward(const Adapters& a, const uint16_t* dy, const uint16_t* x, const float* hidden,
                            const uint16_t* down, const uint16_t* up, const uint16_t* dx_add, uint16_t* dx,
                            float* ddown, float* dup, int N, int K, void* ws, hipStream_t s) {
    Outer o{};
    o.scales = a.scales;
    o.M = a.M;
    o.R = a.R;
    o.L = a.L;
    o.splits = 1;
    o.job[0] = {nullptr, x, ddown, nullptr, a.drop, K, 0};
    o.job[1] = {hidden, dy, dup, nullptr, kNoDrop, N, 0};
    if (a.M == 0) return outer(a, o, s);
    const BackwardRoom room(a.M, N, K, a.R, a.L);
    char* at = static_cast<char*>(ws);
    float* part = reinterpret_cast<float*>(at + room.part);
    float* dh = reinterpret_cast<float*>(at + room.dh);
    int32_t* start = ddown && a.slots ? reinterpret_cast<int32_t*>(at + room.start) : nullptr;
    int32_t* list = start ? reinterpret_cast<int32_t*>(at + room.list) : nullptr;
    wq_status st = shrink(a, dy, up, kNoDrop, part, N, start, list, s);
    if (st == WQ_OK)
        st = expand(a, part, ShrinkPlan(a.M, a.R, a.L, N).splits, down, a.drop, dx_add, dx, ddown ? dh : nullptr, K, s);
    if (st != WQ_OK || !ddown) return st;
    o.splits = room.splits;
    o.start = start;
    o.list = list;
    o.job[0].h = dh;
    o.job[0].part = reinterpret_cast<float*>(at + room.outer0);
    o.job[1].part = reinterpret_cast<float*>(at + room.outer1);
    return outer(a, o, s);
}

}  // namespace wqh
