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
constexpr int kChunk = 128;   // columns of src by which a shrink is split into ranges
constexpr int kShrinkWaves = 8;
constexpr int kCols = 128;    // columns of out and dw of a wavefront: 16 lanes of 8

// Eight fp16 values at p, which need not be aligned to more than one of them
// (odd row lengths): the hardware takes 16-byte accesses at any address.
__device__ __forceinline__ u4 load8(const uint16_t* p) {
    u4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
// Within a window or an adapter, element numbers fit 32 bits (64 rows, or 128
// of the rank, of at most 2^22 columns): a uniform base and a 32-bit offset,
// which the loads take as they are.
__device__ __forceinline__ const uint16_t* off(const uint16_t* base, uint32_t n) {
    return reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(base) + n * 2u);
}
// The last columns of a row of C (at least 8): where a load of eight from
// column c on would pass the row's end it is taken from C - 8 on, and what comes
// before c is shifted out.
__device__ __forceinline__ int held(int c, int C) { return min(c, C - 8); }
__device__ __forceinline__ u4 shifted(u4 v, int c, int C) {
    const int s = c - held(c, C);
    if (s & 1)
        v = u4{__builtin_amdgcn_alignbit(v[1], v[0], 16), __builtin_amdgcn_alignbit(v[2], v[1], 16),
               __builtin_amdgcn_alignbit(v[3], v[2], 16), v[3] >> 16};
    if (s & 2) v = u4{v[1], v[2], v[3], 0};
    if (s & 4) v = u4{v[2], v[3], 0, 0};
    if (s >= 8) v = u4{0, 0, 0, 0};
    return v;
}
// The first n of eight values.
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
// block's range of columns; the wavefronts take pieces of it in turn, the
// next one's loads in flight.  Rows past the adapter's repeat its last one, and rows past
// the rank likewise: they cost no traffic, and what they give is not kept.
template <int MT, int NRT, bool DROP>
__device__ __forceinline__ void shrink_rows(const Shrink& p, int64_t m0, int a, int cnt, int order, int r0, int split,
                                            f4* sum) {
    constexpr int STEPS = MT * NRT > 8 ? 1 : 2, COLS = 32 * STEPS;   // 128 bytes of a row, or what the registers hold
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, g = lane >> 4;
    f4 acc[MT][NRT];
    const uint16_t* const xb = p.src + m0 * p.C;
    const uint16_t* const wb = p.w + int64_t(a) * p.R * p.C;
    const uint64_t eight = uint64_t(m0) * (p.C / 8);
    uint32_t xr[MT], wr[NRT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        xr[t] = uint32_t(__shfl(order, min(16 * t + c16, cnt - 1))) * p.C;
#pragma unroll
        for (int n = 0; n < NRT; ++n) acc[t][n] = f4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int n = 0; n < NRT; ++n) wr[n] = uint32_t(min(r0 + 16 * n + c16, p.R - 1)) * p.C;
    const uint64_t stream = DROP ? wq::drop_stream(p.drop) : 0;

    struct Part {
        u4 x[MT][STEPS], w[NRT][STEPS];
    };
    auto load = [&](int c0, Part& v) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int c = held(c0 + 32 * i + 8 * g, p.C);
#pragma unroll
            for (int n = 0; n < NRT; ++n) v.w[n][i] = load8(off(wb, wr[n] + c));
#pragma unroll
            for (int t = 0; t < MT; ++t) v.x[t][i] = load8(off(xb, xr[t] + c));
        }
    };
    auto multiply = [&](int c0, Part& v) {
        if (c0 + COLS > p.C)
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int c = c0 + 32 * i + 8 * g;
#pragma unroll
                for (int n = 0; n < NRT; ++n) v.w[n][i] = shifted(v.w[n][i], c, p.C);
#pragma unroll
                for (int t = 0; t < MT; ++t) v.x[t][i] = shifted(v.x[t][i], c, p.C);
            }
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if constexpr (DROP) v.x[t][i] = drop8(v.x[t][i], eight + ((xr[t] + c0 + 32 * i + 8 * g) >> 3), p.drop, stream);
#pragma unroll
                for (int n = 0; n < NRT; ++n) acc[t][n] = mfma(v.x[t][i], v.w[n][i], acc[t][n]);
            }
    };
    const int end = int(min(int64_t(split + 1) * p.cps * kChunk, int64_t(p.C)));
    constexpr int NEXT = kShrinkWaves * COLS;
    int c0 = split * p.cps * kChunk + wave * COLS;
    Part v[2];
    if (c0 < end) load(c0, v[0]);
    for (; c0 < end; c0 += 2 * NEXT) {
        if (c0 + NEXT < end) load(c0 + NEXT, v[1]);
        multiply(c0, v[0]);
        if (c0 + 2 * NEXT < end) load(c0 + 2 * NEXT, v[0]);
        if (c0 + NEXT < end) multiply(c0 + NEXT, v[1]);
    }

    // the wavefronts' sums: w and w + 4, then the four in order
    constexpr int HALF = kShrinkWaves / 2;
    auto at = [&](int t, int n, int w) { return ((t * NRT + n) * HALF + w) * 64 + lane; };
    if (wave >= HALF)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < NRT; ++n) sum[at(t, n, wave - HALF)] = acc[t][n];
    __syncthreads();
    if (wave < HALF)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < NRT; ++n) sum[at(t, n, wave)] += acc[t][n];
    __syncthreads();
    const int RP = NRT * 16 * p.rchunks;
    for (int e = wave; e < MT * NRT; e += kShrinkWaves) {
        const int t = e / NRT, n = e % NRT, r = r0 + 16 * n + c16;
        f4 v = sum[at(t, n, 0)];
#pragma unroll
        for (int i = 1; i < HALF; ++i) v += sum[at(t, n, i)];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * t + 4 * g + i;
            const int64_t m = m0 + __shfl(order, row);
            if (row < cnt)
                p.part[(int64_t(split) * p.M + m) * RP + r] = r < p.R ? DROP ? v[i] * p.drop.keep : v[i] : 0.f;
        }
    }
    __syncthreads();
}

// Blocks: for a window, its ranges of columns (neighbouring blocks: the XCDs
// take them in turn, so that each holds its own range of every adapter in L2),
// the rank's 64s, and Z shares of its adapters.
template <int NRT, bool DROP>
__global__ __launch_bounds__(64 * kShrinkWaves) void shrink_kernel(const Shrink p, int64_t first) {
    __shared__ f4 sum[4 * NRT * 64 * (kShrinkWaves / 2)];
    int64_t b = first + blockIdx.x;
    if (b >= p.blocks) {
        list_rows(p, (b - p.blocks) * kShrinkWaves + (threadIdx.x >> 6));
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

// h of an adapter's rows, four threads to a row: summed over the ranges, scaled
// into fp16's range row by row and split in two.
template <int RP>
__device__ __forceinline__ void expand_parts(const Expand& p, int64_t m0, int cnt, int order, bool keep_sum,
                                             uint16_t* parts, float* back) {
    typedef ExpandTile<RP> T;
    const int row = threadIdx.x >> 2, q = threadIdx.x & 3;
    const int64_t m = m0 + __shfl(order, min(row, cnt - 1));
    if (row >= (cnt + 15) / 16 * 16) return;   // (whole wavefronts)
    f4 v[RP / 16];
#pragma unroll
    for (int i = 0; i < RP / 16; ++i) v[i] = f4{0.f, 0.f, 0.f, 0.f};
    const float* h = p.part + m * RP + q * (RP / 4);
    const int64_t next = int64_t(p.M) * RP;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s, h += next)
#pragma unroll
        for (int i = 0; i < RP / 16; ++i) v[i] += *reinterpret_cast<const f4*>(h + 4 * i);
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
    if (keep_sum && row < cnt)
#pragma unroll
        for (int i = 0; i < RP / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = q * (RP / 4) + 4 * i + j;
                if (r < p.R) p.sum[m * p.R + r] = v[i][j];
            }
}

// One adapter's rows, up to 16 MT, against the block's columns.
template <int RP, int MT, bool DROP>
__device__ __forceinline__ void expand_rows(const Expand& p, int64_t m0, int a, int cnt, int order, int cb,
                                            uint16_t* parts, float* back) {
    typedef ExpandTile<RP> T;
    constexpr int G = MT > 2 ? 2 : MT;   // 16-row tiles whose old values are loaded at a time
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, g = lane >> 4;
    const int wave0 = (cb * p.span * 4 + wave) * kCols;   // the wavefront's first column
    const uint64_t stream = DROP ? wq::drop_stream(p.drop) : 0, eight = uint64_t(m0) * (p.C / 8);
    const uint16_t* const wb = p.w + int64_t(a) * p.R * p.C;
    const uint16_t* const ab = p.add + m0 * p.C;
    uint16_t* const ob = p.out + m0 * p.C;
    uint32_t row[MT * 4];   // where the lane's rows begin, from the window's first on
#pragma unroll
    for (int i = 0; i < MT * 4; ++i)
        row[i] = uint32_t(__shfl(order, min(16 * (i >> 2) + 4 * g + (i & 3), cnt - 1))) * p.C;
    constexpr bool AHEAD = RP <= 32;   // w is loaded before h is ready, and a column tile ahead
    u4 raw[AHEAD ? T::KB : 1][8], old[G * 4];
    auto load_piece = [&](u4 (&v)[8], int k, int c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = T::BOTH ? 8 * (g & 1) + i : 32 * k + 8 * g + i;
            v[i] = load8(off(wb, uint32_t(min(r, p.R - 1)) * p.C + held(c, p.C)));
        }
    };
    auto load_w = [&](int c) {
        if constexpr (AHEAD)
#pragma unroll
            for (int k = 0; k < T::KB; ++k) load_piece(raw[k], k, c);
    };
    auto load_old = [&](int t0, int c) {
        if (!p.add) return;
#pragma unroll
        for (int i = 0; i < G * 4; ++i) old[i] = load8(off(ab, row[t0 * 4 + i] + held(c, p.C)));
    };
    // one column tile of the wavefront: its loads are in flight
    auto tile = [&](int c, bool full, float s, auto&& next) {
        u4 w[T::KB][8];
#pragma unroll
        for (int k = 0; k < T::KB; ++k) {
            u4(&v)[8] = raw[AHEAD ? k : 0];
            if constexpr (!AHEAD) load_piece(v, k, c);
            if (p.R < RP) {   // rows past the rank: zeros, as h is there
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if ((T::BOTH ? 8 * (g & 1) + i : 32 * k + 8 * g + i) >= p.R) v[i] = u4{0, 0, 0, 0};
            }
            if (!full)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = shifted(v[i], c, p.C);
            transpose8(v, w[k]);
        }
        next();
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if (t > 0 && t % G == 0) {
                __builtin_amdgcn_sched_barrier(0);
                load_old(t, c);
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
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = acc[j][i] * inverse[i] * s;
                if constexpr (DROP) {
                    const u4 d = wq::philox(eight + ((row[t * 4 + i] + c) >> 3), stream, p.drop.key0, p.drop.key1);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = wq::kept(d, j, p.drop.t) ? f[j] : 0.f;
                }
                if (p.add) {
                    u4 o = old[t % G * 4 + i];
                    if (!full) o = shifted(o, c, p.C);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] += wq::h2f(uint16_t(o[j >> 1] >> (16 * (j & 1))));
                }
                u4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = wq::f2h(f[2 * j]) | uint32_t(wq::f2h(f[2 * j + 1])) << 16;
                if (16 * t + 4 * g + i < cnt) {
                    uint16_t* to = const_cast<uint16_t*>(off(ob, row[t * 4 + i] + c));
                    if (full)
                        __builtin_memcpy(to, &v, 16);
                    else
                        store8_part(to, v, p.C - c);
                }
            }
        }
    };

    const bool any = p.out && wave0 < p.C;
    if (any) {
        load_w(wave0 + 8 * c16);
        load_old(0, wave0 + 8 * c16);
    }
    expand_parts<RP>(p, m0, cnt, order, p.sum && cb == 0, parts, back);
    __syncthreads();
    if (any) {
        const float s = p.scales[a] * (DROP ? p.drop.keep : 1.f);
        for (int ct = 0; ct < p.span; ++ct) {
            const int c0 = wave0 + ct * 4 * kCols, c = c0 + 8 * c16;
            if (c0 >= p.C) break;
            const int n0 = c0 + 4 * kCols;
            if (ct) load_old(0, c);
            tile(c, c0 + kCols <= p.C, s, [&] {
                if (ct + 1 < p.span && n0 < p.C) load_w(n0 + 8 * c16);
            });
        }
    }
    __syncthreads();
}

template <int RP, bool DROP>
__global__ __launch_bounds__(256, RP > 64 ? 1 : 2) void expand_kernel(const Expand p, int64_t total, int64_t first) {
    __shared__ __attribute__((aligned(16))) uint16_t parts[kWindow * ExpandTile<RP>::STRIDE];
    __shared__ __attribute__((aligned(16))) float back[kWindow];
    const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
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

    each_adapter(slot, z, p.Z, [&](int a, int cnt, int order) {
        if (cnt <= 16)
            expand_rows<RP, 1, DROP>(p, m0, a, cnt, order, cb, parts, back);
        else if (cnt <= 32)
            expand_rows<RP, 2, DROP>(p, m0, a, cnt, order, cb, parts, back);
        else
            expand_rows<RP, 4, DROP>(p, m0, a, cnt, order, cb, parts, back);
    });

    const int col0 = (cb * p.span * 4 + int(threadIdx.x >> 6)) * kCols + 8 * c16;
    // rows without an adapter
    const uint64_t none = z == 0 ? __ballot(slot < 0 && m0 + lane < p.M) : 0;
    if (!none) return;
    const int cnt = __builtin_popcountll(none), order = compact(none);
    if (p.out && p.out != p.add)
        for (int ct = 0; ct < p.span; ++ct) {
            const int c = col0 + ct * 4 * kCols;
            if (c - 8 * c16 >= p.C) break;
            for (int row = 0; row < cnt; row += 4) {
                const int64_t m = m0 + __shfl(order, row + g);
                if (row + g >= cnt) continue;
                u4 v{0, 0, 0, 0};
                if (p.add) v = shifted(load8(p.add + m * p.C + held(c, p.C)), c, p.C);
                store8_part(p.out + m * p.C + c, v, p.C - c);
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
    const int c = tile * kCols + 8 * c16, left = j.C - c;
    const bool full = (tile + 1) * kCols <= j.C, drop = j.drop.t != 0;
    const uint64_t stream = drop ? wq::drop_stream(j.drop) : 0;
    const int steps = (cnt + 31) / 32;
    const int end = int(int64_t(split + 1) * steps / p.splits);
    // fragment t holds r0 + NRT (l % 16) + t, a lane's r side by side; for those past
    // the rank others are taken: what they give is not kept
    const int held_r = min(r0 + NRT * c16, p.R - NRT);
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
        int64_t m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // (rows past the adapter's repeat its last one)
            const int n = min(i0 + i, cnt - 1);
            m[i] = p.list ? p.list[at + n] : n;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = load8(j.src + m[i] * j.C + held(c, j.C));
            __builtin_memcpy(h[i], j.h + m[i] * p.R + held_r, 4 * NRT);
        }
        if (p.R % NRT) {   // a lane whose r's end inside NRT of them took the rank's last NRT
            const int by = r0 + NRT * c16 - held_r;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v[NRT];
#pragma unroll
                for (int t = 0; t < NRT; ++t) {
                    v[t] = h[i][t];
#pragma unroll
                    for (int k = 1; t + k < NRT; ++k) v[t] = by == k ? h[i][t + k] : v[t];
                }
#pragma unroll
                for (int t = 0; t < NRT; ++t) h[i][t] = v[t];
            }
        }
        if (!full)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = shifted(x[i], c, j.C);
        if (drop)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = drop8(x[i], (uint64_t(m[i]) * j.C + c) >> 3, j.drop, stream);
        if (st * 32 + 32 > cnt)   // they count as zeros
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i >= cnt) {
                    x[i] = u4{0, 0, 0, 0};
#pragma unroll
                    for (int t = 0; t < NRT; ++t) h[i][t] = 0.f;
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
    if (q >= size || (second && j.C < 8)) return;
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

// ------------------------------------------------------- narrow projections ----
//
// With fewer than eight columns rows are shorter than a load.  One thread to an
// element; the products have at most seven columns.

// part[0][m][r], columns past R zero, of src [M][C].
__global__ __launch_bounds__(256) void narrow_shrink_kernel(const Shrink p, int RP, int64_t first) {
    const int64_t q = (first + blockIdx.x) * 256 + threadIdx.x, m = q / RP;
    const int r = int(q % RP);
    if (m >= p.M) return;
    const int a = slot_of(p.slots, m, p.M, p.L);
    float v = 0.f;
    if (a >= 0 && r < p.R)
        for (int c = 0; c < p.C; ++c)
            v += wq::h2f(p.src[m * p.C + c]) * wq::h2f(p.w[(int64_t(a) * p.R + r) * p.C + c]);
    p.part[q] = v;
}
__global__ __launch_bounds__(64 * kShrinkWaves) void list_kernel(const Shrink p, int64_t first) {
    list_rows(p, (first + blockIdx.x) * kShrinkWaves + (threadIdx.x >> 6));
}

// out of C columns; thread 0 of a row's columns also leaves the row's sums.
__global__ __launch_bounds__(256) void narrow_expand_kernel(const Expand p, int RP, int64_t first) {
    const int64_t q = (first + blockIdx.x) * 256 + threadIdx.x, m = q / p.C;
    const int c = int(q % p.C);
    if (m >= p.M) return;
    const int a = slot_of(p.slots, m, p.M, p.L);
    float v = 0.f;
    for (int r = 0; r < p.R; ++r) {
        float h = 0.f;
        if (a >= 0) {
            for (int s = 0; s < p.splits; ++s) h += p.part[(int64_t(s) * p.M + m) * RP + r];
            v += h * wq::h2f(p.w[(int64_t(a) * p.R + r) * p.C + c]);
        }
        if (p.sum && c == 0) p.sum[m * p.R + r] = h;
    }
    if (a >= 0) v *= p.scales[a];
    p.out[q] = p.add ? a >= 0 ? wq::f2h(wq::h2f(p.add[q]) + v) : p.add[q] : wq::f2h(v);
}

// One gradient of C columns, a wavefront to an element.
__global__ __launch_bounds__(64) void narrow_outer_kernel(const Outer p, int64_t first) {
    const OuterJob& j = p.job[1];
    const int64_t q = first + blockIdx.x, ar = q / j.C;
    const int c = int(q % j.C), a = int(ar / p.R), r = int(ar % p.R);
    const int at = p.start ? p.start[a] : 0, cnt = p.start ? p.start[a + 1] - at : a == 0 ? p.M : 0;
    float v = 0.f;
    for (int i = threadIdx.x; i < cnt; i += 64) {
        const int64_t m = p.list ? p.list[at + i] : i;
        v += j.h[m * p.R + r] * wq::h2f(j.src[m * j.C + c]);
    }
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    if (threadIdx.x == 0) j.dw[q] = cnt ? v * p.scales[a] : 0.f;
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
    const int lists = start ? div_up(a.L, kShrinkWaves) : 0;
    if (C < 8) {   // (N: K is 32 at least, so nothing is dropped)
        const wq_status st = pieces((int64_t(a.M) * RP + 255) / 256, [&](unsigned blocks, int64_t first) {
            narrow_shrink_kernel<<<blocks, 256, 0, s>>>(p, RP, first);
        });
        if (st != WQ_OK) return st;
        return pieces(lists, [&](unsigned blocks, int64_t first) {
            list_kernel<<<blocks, 64 * kShrinkWaves, 0, s>>>(p, first);
        });
    }
    const int64_t all = p.blocks + lists;
    return pieces(all, [&](unsigned blocks, int64_t first) {
        auto go = [&](auto n) {
            if (d.t)
                shrink_kernel<decltype(n)::value, true><<<blocks, 64 * kShrinkWaves, 0, s>>>(p, first);
            else
                shrink_kernel<decltype(n)::value, false><<<blocks, 64 * kShrinkWaves, 0, s>>>(p, first);
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
    if (out && C < 8)
        return pieces((int64_t(a.M) * C + 255) / 256, [&](unsigned blocks, int64_t first) {
            narrow_expand_kernel<<<blocks, 256, 0, s>>>(p, padded_rank(a.R), first);
        });
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
    const bool narrow = p.job[1].C < 8;
    if (narrow) {
        const wq_status st = pieces(int64_t(a.L) * a.R * p.job[1].C, [&](unsigned blocks, int64_t first) {
            narrow_outer_kernel<<<blocks, 64, 0, s>>>(p, first);
        });
        if (st != WQ_OK) return st;
    }
    wq_status st = pieces(p.blocks0 + (narrow ? 0 : per * p.job[1].tiles), [&](unsigned blocks, int64_t first) {
        if (RP == 16)
            outer_kernel<1><<<blocks, 256, 0, s>>>(p, first);
        else if (RP == 32)
            outer_kernel<2><<<blocks, 256, 0, s>>>(p, first);
        else
            outer_kernel<4><<<blocks, 256, 0, s>>>(p, first);
    });
    if (st != WQ_OK || p.splits == 1) return st;
    const int64_t n0 = (int64_t(a.L) * a.R * p.job[0].C + 3) / 4 * 4, n1 = narrow ? 0 : int64_t(a.L) * a.R * p.job[1].C;
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
