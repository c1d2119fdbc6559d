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
constexpr int kShrinkWaves = 8, kDirectWaves = 8;
constexpr int kDirectM = 16, kDirectK = 4096;   // the one-launch form's: a fragment's rows, K in a block's registers
constexpr int kPad = 128;     // numbers behind the last list: a round of the gradients reads whole ones
constexpr int kCols = 128;    // columns of out and dw of a wavefront: 16 lanes of 8

// Eight fp16 values at p, which need not be aligned to more than one of them
// (odd row lengths): the hardware takes 16-byte accesses at any address.
__device__ __forceinline__ u4 load8(const uint16_t* p) {
    u4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
__device__ __forceinline__ void store8(uint16_t* p, u4 v) { __builtin_memcpy(p, &v, 16); }

// The wavefront's number, as the scalar that it is: the matrix instructions do not
// heed the execution mask, so what leads to them has to branch.
__device__ __forceinline__ int wave_of() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Within a window or an adapter, element numbers fit 32 bits (64 rows, or 128
// of the rank, of at most 2^22 columns): a uniform base and a 32-bit offset,
// which the loads take as they are.
__device__ __forceinline__ const uint16_t* off(const uint16_t* base, uint32_t n) {
    return reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(base) + n * 2u);
}
__device__ __forceinline__ uint16_t* off(uint16_t* base, uint32_t n) {
    return reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(base) + n * 2u);
}

// Where the eight columns of a lane begin that nominally begin at c: the last
// eight of a row of C (at least 8) take the place of any that would pass its
// end.  Columns held twice are written twice, the same value, or masked.
__device__ __forceinline__ int held(int c, int C) { return min(c, C - 8); }

__device__ __forceinline__ f4 mfma(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// Rows 8 g + i of a fragment's k dimension as 8 loads of 8 neighbouring
// columns, to the fragments of those columns: fragment j holds column j of the
// lane's eight, so a lane ends up with eight neighbouring columns of the result.
__device__ __forceinline__ void transpose8(const u4 (&row)[8], u4 (&frag)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            frag[j][q] = __builtin_amdgcn_perm(row[2 * q + 1][j >> 1], row[2 * q][j >> 1],
                                               j & 1 ? 0x07060302u : 0x05040100u);
}

// Lane l's row of a window: its slot, -1 for one without an adapter.
__device__ __forceinline__ int slot_of(const int32_t* slots, int64_t m, int M, int L) {
    if (m >= M) return -1;
    const int s = slots ? slots[m] : 0;
    return unsigned(s) < unsigned(L) ? s : -1;
}
__device__ __forceinline__ int lanes_below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi(uint32_t(mask >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(mask), 0));
}
// The lanes in `mask` first, in order, then the others: lane i gets the i-th's number.
__device__ __forceinline__ int compact(uint64_t mask) {
    const int lane = threadIdx.x & 63, below = lanes_below(mask);
    const int to = mask >> lane & 1 ? below : __builtin_popcountll(mask) + lane - below;
    return __builtin_amdgcn_ds_permute(to * 4, lane);
}

// Calls work(adapter, rows, order) for the window's adapters z, z + Z, ... in
// order of appearance; order: the adapter's rows first.
template <class Work>
__device__ __forceinline__ void each_adapter(int slot, int z, int Z, const Work& work) {
    uint64_t todo = __ballot(slot >= 0);
    for (int n = 0; todo; n = n + 1 == Z ? 0 : n + 1) {
        const int a = __builtin_amdgcn_readlane(slot, __builtin_ctzll(todo));
        const uint64_t mine = __ballot(slot == a);
        todo &= ~mine;
        if (n == z) work(a, __builtin_popcountll(mine), compact(mine));
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
// The largest finite magnitude of v (0 where there is none).  Infinities and NaN
// sort above every number, so that one comparison tells whether to look again.
template <int N>
__device__ __forceinline__ float largest(const float (&v)[N], bool& odd) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) most = max(most, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    odd = most >= 0x7F800000u;
    if (odd) {
        most = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t m = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
            most = max(most, m < 0x7F800000u ? m : 0u);
        }
    }
    return __builtin_bit_cast(float, most);
}
typedef float f2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_h(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, wq::h2));
}
// scale a and scale b (a power of two) as sums of two fp16 numbers each: the
// second is what the first leaves, one multiply-add.  The matrix instructions that
// take fp16 weights as they are take fp16 beside them; two parts leave 2^-22 of
// a value (2^-25 where that is more, 2^-38 of the largest), near fp32's own 2^-24,
// for twice the instructions, and a third part would be half as many again.
__device__ __forceinline__ void split_h(float a, float b, float scale, uint32_t& hi, uint32_t& lo) {
    hi = pack_h(a * scale, b * scale);
    const wq::h2 h = wq::as_h2(hi);
    lo = pack_h(__builtin_fmaf(a, scale, -float(h[0])), __builtin_fmaf(b, scale, -float(h[1])));
}
// An infinity of h leaves NaN in the rest: zero instead.
__device__ __forceinline__ uint32_t without_rest(uint32_t hi, uint32_t lo) {
    if ((hi & 0x7FFFu) == 0x7C00u) lo &= 0xFFFF0000u;
    if ((hi & 0x7FFF0000u) == 0x7C000000u) lo &= 0xFFFFu;
    return lo;
}

// An infinity of the other operand makes NaN of a rest that is zero or of the
// other sign, where h times it is an infinity.  So sums that are not finite are made
// again without the split.  Whether a lane holds one: IEEE 754's maximum keeps NaN, and is
// one instruction for two values (16 to a 16 x 128 tile; all of this takes up to
// 0.3 us of a decode call, 1% of a large one).
__device__ __forceinline__ bool finite(float v) { return __builtin_fabsf(v) < __builtin_inff(); }
template <int N>
__device__ __forceinline__ bool any_odd(const f4 (&v)[N]) {
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) most = __builtin_elementwise_maximum(most, __builtin_fabsf(v[j][i]));
    return __ballot(!finite(most)) != 0;
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
    int32_t* list;         // [M + kPad], zeros behind the rows
    int lists;             // layers of y that make them
    int window0;           // of this launch
};

// Lists of rows by adapter: a block per adapter, next to the product's.  Its
// wavefronts take a range of rows each, count the rows of lower adapters (their
// sum is the list's start) and their own, and write those in order.
__device__ __forceinline__ void list_rows(const Shrink& p, int a, int* counts) {
    const int lane = threadIdx.x & 63, wave = wave_of();
    if (a >= p.L) return;
    constexpr int U = 4;
    const int each = (p.M + 64 * U * kShrinkWaves - 1) / (64 * U * kShrinkWaves) * 64 * U;
    const int64_t first = int64_t(wave) * each, end = min(first + each, int64_t(p.M));
    int s[U];
    auto load = [&](int64_t m) {   // -1 where there is no row
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = m + 64 * u + lane < end ? p.slots[m + 64 * u + lane] : -1;
    };
    int less = 0, mine = 0;
#pragma unroll 1
    for (int64_t m = first; m < end; m += 64 * U) {
        load(m);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            less += __builtin_popcountll(__ballot(unsigned(s[u]) < unsigned(a)));
            mine += __builtin_popcountll(__ballot(s[u] == a));
        }
    }
    if (lane == 0) {
        counts[wave] = less;
        counts[kShrinkWaves + wave] = mine;
    }
    __syncthreads();
    int start = 0, all = 0, before = 0;
    for (int w = 0; w < kShrinkWaves; ++w) {
        start += counts[w];
        if (w == wave) before = all;
        all += counts[kShrinkWaves + w];
    }
    if (threadIdx.x == 0) {
        p.start[a] = start;
        if (a == p.L - 1) p.start[p.L] = start + all;
    }
    if (a == p.L - 1 && threadIdx.x < kPad) p.list[start + all + threadIdx.x] = 0;
    if (!mine) return;
    int at = start + before;
#pragma unroll 1
    for (int64_t m = first; m < end; m += 64 * U) {
        load(m);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint64_t mask = __ballot(s[u] == a);
            if (s[u] == a) p.list[at + lanes_below(mask)] = int(m + 64 * u + lane);
            at += __builtin_popcountll(mask);
        }
    }
}

// One adapter's rows of a window, up to 16 MT, against 16 NRT of its rank's
// rows, over the block's range of columns; the wavefronts take pieces of it in
// turn, with AHEAD the next one's loads in flight.  Rows past the adapter's repeat its
// last one, and rows past the rank likewise: they cost no traffic, and what
// they give is not kept.
template <int MT, int NRT, bool DROP, bool AHEAD>
__device__ __forceinline__ void shrink_rows(const Shrink& p, int64_t m0, int a, int cnt, int order, int r0, int split,
                                            f4* sum) {
    constexpr int STEPS = MT * NRT > 8 ? 1 : 2, COLS = 32 * STEPS;   // 128 bytes of a row, or what the registers hold
    const int lane = threadIdx.x & 63, wave = wave_of(), c16 = lane & 15, g = lane >> 4;
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
    const int end = int(min(int64_t(split + 1) * p.cps * kChunk, int64_t(p.C)));
    constexpr int NEXT = kShrinkWaves * COLS;
    int c0 = split * p.cps * kChunk + wave * COLS;
    Part v, next;
    if (c0 < end) load(c0, v);
#pragma unroll 1
    for (; c0 < end; c0 += NEXT) {
        if (AHEAD && c0 + NEXT < end) load(c0 + NEXT, next);
        if (c0 + COLS > p.C)   // columns that other lanes hold too: zeros on both sides
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int twice = c0 + 32 * i + 8 * g - held(c0 + 32 * i + 8 * g, p.C);
                u4 mask;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    mask[q] = (twice <= 2 * q ? 0xFFFFu : 0u) | (twice <= 2 * q + 1 ? 0xFFFF0000u : 0u);
#pragma unroll
                for (int n = 0; n < NRT; ++n) v.w[n][i] &= mask;
#pragma unroll
                for (int t = 0; t < MT; ++t) v.x[t][i] &= mask;
            }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            if constexpr (DROP) {
                uint64_t at[MT];
                u4 keep[MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) at[t] = eight + ((xr[t] + c0 + 32 * i + 8 * g) >> 3);
                wq::keep8(at, p.drop, stream, keep);
#pragma unroll
                for (int t = 0; t < MT; ++t) v.x[t][i] &= keep[t];
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int n = 0; n < NRT; ++n) acc[t][n] = mfma(v.x[t][i], v.w[n][i], acc[t][n]);
        }
        if (AHEAD)
            v = next;
        else if (c0 + NEXT < end)
            load(c0 + NEXT, v);
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
#pragma unroll 1
    for (int e = wave; e < MT * NRT; e += kShrinkWaves) {
        const int t = e / NRT, n = e % NRT, r = r0 + 16 * n + c16;
        f4 v = sum[at(t, n, 0)];
#pragma unroll
        for (int i = 1; i < HALF; ++i) v += sum[at(t, n, i)];
        float* to = p.part + (int64_t(split) * p.M + m0) * RP + r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * t + 4 * g + i, m = __shfl(order, row & 63);
            if (row < cnt) to[m * RP] = r < p.R ? DROP ? v[i] * p.drop.keep : v[i] : 0.f;
        }
    }
    __syncthreads();
}

// Blocks: x the ranges of columns (the XCDs take neighbours in turn, so that
// each holds its own range of every adapter in L2), y the window, behind the
// layers that make the lists, z the rank's 64s and Z shares of the window's
// adapters.
//
// ONE: 16 rows at a time and one piece in flight, for decode batches of many
// adapters: that leaves registers for twice the wavefronts, and those blocks
// wait for a few short loads.
//
// Bound by latency below some 2000 rows, then by memory, with dropout by the
// masks' vector instructions.  Measured, us, all rows of one adapter and in five or
// four runs (a window at a run's border takes its adapters one after the other, and
// the launch lasts as long as that block): 2048 rows, C = 4096, rank 16, 6.0 to 6.7
// and 8.6 to 9.7; 4096 rows, rank 64, 12.2 and 18.9 to 22.2; with dropout, of one
// adapter, 15.2.  128 rows of 24 adapters, C = 11008, rank 64, 14.4 to 15.2: the 34 MB
// of weights come from memory once, a block takes two or three adapters in series.
// Rows of odd length are read by accesses that are aligned to 2 bytes, at half the
// rate: 311 rows of C = 5001, rank 8, 9.1, of 5004 4.7, with lists or without.
template <int NRT, bool DROP, bool ONE>
__global__ __launch_bounds__(64 * kShrinkWaves, ONE ? 4 : 2) void shrink_kernel(const Shrink p) {
    constexpr int MT = ONE ? 1 : 4;
    __shared__ f4 sum[MT * NRT * 64 * (kShrinkWaves / 2)];
    if (int(blockIdx.y) < p.lists) {
        list_rows(p, int((blockIdx.y * gridDim.z + blockIdx.z) * gridDim.x + blockIdx.x), reinterpret_cast<int*>(sum));
        return;
    }
    const int bz = blockIdx.z;
    const int split = blockIdx.x, r0 = p.rchunks > 1 ? (bz & 1) * 64 : 0, z = p.rchunks > 1 ? bz >> 1 : bz;
    const int64_t m0 = int64_t(p.window0 + int(blockIdx.y) - p.lists) * kWindow;
    const int slot = slot_of(p.slots, m0 + (threadIdx.x & 63), p.M, p.L);
    each_adapter(slot, z, p.Z, [&](int a, int cnt, int order) {
#pragma unroll 1
        for (; cnt > 0; cnt -= 16 * MT) {
            shrink_rows<MT, NRT, DROP, !ONE>(p, m0, a, min(cnt, 16 * MT), order, r0, split, sum);
            order = __shfl(order, (threadIdx.x + 16 * MT) & 63);
        }
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
    int Z, halves;         // blocks that share a window's adapters; and an adapter's rows
    int span;              // a block's columns: span * 512
    int window0;           // of this launch
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
    if (row >= (cnt + 15) / 16 * 16) return;   // (whole wavefronts)
    const int64_t m = m0 + __shfl(order, min(row, cnt - 1));
    f4 v[RP / 16];
#pragma unroll
    for (int i = 0; i < RP / 16; ++i) v[i] = f4{0.f, 0.f, 0.f, 0.f};
    const float* h = p.part + m * RP + q * (RP / 4);
    const int64_t next = int64_t(p.M) * RP;
    constexpr int U = RP > 32 ? 2 : 4;
#pragma unroll U
    for (int s = 0; s < p.splits; ++s, h += next)
#pragma unroll
        for (int i = 0; i < RP / 16; ++i) v[i] += *reinterpret_cast<const f4*>(h + 4 * i);
    float all[RP / 4];
#pragma unroll
    for (int i = 0; i < RP / 4; ++i) all[i] = v[i >> 2][i & 3];
    bool odd;
    float most = largest(all, odd);
    most = __builtin_fmaxf(most, __shfl_xor(most, 1));
    most = __builtin_fmaxf(most, __shfl_xor(most, 2));
    float inverse;
    const float scale = to_range(most, 13, inverse);
    if (q == 0) back[row] = inverse;
    uint32_t* to = reinterpret_cast<uint32_t*>(parts + row * T::STRIDE + q * (RP / 4));
#pragma unroll
    for (int i = 0; i < RP / 8; ++i) {
        uint32_t hi, lo;
        split_h(all[2 * i], all[2 * i + 1], scale, hi, lo);
        to[i] = hi;
        to[RP / 2 + i] = odd ? without_rest(hi, lo) : lo;
    }
    if (keep_sum && row < cnt) {
        float* at = p.sum + m * p.R;
#pragma unroll
        for (int i = 0; i < RP / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = q * (RP / 4) + 4 * i + j;
                if (r < p.R) at[r] = v[i][j];
            }
    }
}

// 32 rows of w (16, twice, where both parts share a fragment) at the lane's eight
// columns; those past the rank repeat its last one.
template <int RP>
__device__ __forceinline__ void load_w(u4 (&v)[8], const uint16_t* wb, int k, int c, int R, int C) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = ExpandTile<RP>::BOTH ? 8 * (g & 1) + i : 32 * k + 8 * g + i;
        v[i] = load8(off(wb, uint32_t(min(r, R - 1)) * C + c));
    }
}
// ... into fragments, with zeros past the rank, as h has there.
template <int RP>
__device__ __forceinline__ void make_w(u4 (&v)[8], u4 (&w)[8], int k, int R) {
    const int g = (threadIdx.x & 63) >> 4;
    if (R < RP) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((ExpandTile<RP>::BOTH ? 8 * (g & 1) + i : 32 * k + 8 * g + i) >= R) v[i] = u4{0, 0, 0, 0};
    }
    transpose8(v, w);
}

// 16 rows of h (their parts) times the wavefront's 128 columns of w, onto their
// old values.  at: where the lane's four rows and columns begin, from ob on; c0
// the tile's first column, c the lane's; n: rows of the 16 that are.
template <int RP, bool DROP>
__device__ __forceinline__ void expand_tile(const uint16_t* parts, const float* back, const u4 (&w)[ExpandTile<RP>::KB][8],
                                            const u4 (&old)[4], float s, const uint32_t (&at)[4], uint16_t* ob, int c0,
                                            int c, int C, int n, const Drop& d, uint64_t stream, uint64_t eight) {
    typedef ExpandTile<RP> T;
    const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
    f4 acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = f4{0.f, 0.f, 0.f, 0.f};
    const uint16_t* h = parts + c16 * T::STRIDE + 8 * g;
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
    // The first parts alone (twice where both share an instruction) have h's signs, and
    // their sum is the same infinity or NaN, or it is finite: then the two parts' sum had
    // left fp32's range.
    if (any_odd(acc)) {
        h = parts + c16 * T::STRIDE + 8 * (T::BOTH ? g & 1 : g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f4 t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < T::KB; ++k) t = mfma(*reinterpret_cast<const u4*>(h + 32 * k), w[k][j], t);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = finite(t[i]) ? acc[j][i] : t[i];
        }
    }
    u4 keep[4];
    if constexpr (DROP) {
        uint64_t m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = eight + (at[i] >> 3);
        wq::keep8(m, d, stream, keep);
    }
    const f4 inverse = *reinterpret_cast<const f4*>(back + 4 * g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (a power of two: exact but where the result is below fp16's numbers anyway)
        const float f = inverse[i] * s;
        u4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const wq::h2 o = wq::as_h2(old[i][j]);
            v[j] = pack_h(__builtin_fmaf(acc[2 * j][i], f, float(o[0])),
                          __builtin_fmaf(acc[2 * j + 1][i], f, float(o[1])));
        }
        if constexpr (DROP) v = (v & keep[i]) | (old[i] & ~keep[i]);
        if (4 * g + i >= n) continue;
        if (C - 8 >= c0) {
            store8(off(ob, at[i]), v);
        } else {   // the last, fewer than eight columns: those before c0 are another tile's
#pragma unroll
            for (int j = 1; j < 8; ++j)
                if (c + j >= c0) off(ob, at[i])[j] = uint16_t(v[j >> 1] >> (16 * (j & 1)));
        }
    }
}

// One adapter's rows against the block's columns.
template <int RP, bool DROP, bool ADD>
__device__ __forceinline__ void expand_rows(const Expand& p, int64_t m0, int a, int cnt, int order, uint16_t* parts,
                                            float* back) {
    typedef ExpandTile<RP> T;
    const int lane = threadIdx.x & 63, wave = wave_of(), c16 = lane & 15, g = lane >> 4, cb = blockIdx.y;
    const uint64_t stream = DROP ? wq::drop_stream(p.drop) : 0, eight = uint64_t(m0) * (p.C / 8);
    const uint16_t* const wb = p.w + int64_t(a) * p.R * p.C;
    const uint16_t* const ab = p.add + m0 * p.C;
    uint16_t* const ob = p.out + m0 * p.C;
    const int wave0 = (cb * p.span * 4 + wave) * kCols;   // the wavefront's first column
    const int tiles = (cnt + 15) / 16;
    constexpr bool AHEAD = RP <= 32;   // w and the first old values are loaded before h is ready
    u4 raw[AHEAD ? T::KB : 1][8], old[4], fetched[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) old[i] = u4{0, 0, 0, 0};
    auto load_ahead = [&](int c) {
        if constexpr (AHEAD)
#pragma unroll
            for (int k = 0; k < T::KB; ++k) load_w<RP>(raw[k], wb, k, c, p.R, p.C);
    };
    // where row 16 t + 4 g + i begins, from the window's first on
    auto row_at = [&](int t, int i) { return uint32_t(__shfl(order, min(16 * t + 4 * g + i, cnt - 1))) * p.C; };
    auto load_old = [&](u4 (&v)[4], int t, int c) {
        if constexpr (ADD)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = load8(off(ab, row_at(t, i) + c));
    };

    const bool any = p.out && wave0 < p.C;
    if (any) {
        const int c = held(wave0 + 8 * c16, p.C);
        load_ahead(c);
        load_old(old, 0, c);
    }
    expand_parts<RP>(p, m0, cnt, order, p.sum && cb == 0, parts, back);
    __syncthreads();
    if (any) {
        const float s = p.scales[a] * (DROP ? p.drop.keep : 1.f);
#pragma unroll 1
        for (int ct = 0; ct < p.span; ++ct) {
            const int c0 = wave0 + ct * 4 * kCols, c = held(c0 + 8 * c16, p.C);
            if (c0 >= p.C) break;
            if (ct) load_ahead(c);
            const bool last = ct + 1 == p.span || c0 + 4 * kCols >= p.C;
            const int after = last ? c : held(c0 + 4 * kCols + 8 * c16, p.C);   // the next tile's column
            u4 w[T::KB][8];
#pragma unroll
            for (int k = 0; k < T::KB; ++k) {
                u4(&v)[8] = raw[AHEAD ? k : 0];
                if constexpr (!AHEAD) load_w<RP>(v, wb, k, c, p.R, p.C);
                make_w<RP>(v, w[k], k, p.R);
            }
#pragma unroll 1
            for (int t = 0; t < tiles; ++t) {
                // the next tile's old values (the very last one's again: a branch
                // would end in a wait for them)
                load_old(fetched, t + 1 < tiles ? t + 1 : last ? t : 0, t + 1 < tiles ? c : after);
                uint32_t at[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) at[i] = row_at(t, i) + c;
                expand_tile<RP, DROP>(parts + 16 * t * T::STRIDE, back + 16 * t, w, old, s, at, ob, c0, c, p.C,
                                      cnt - 16 * t, p.drop, stream, eight);
                if constexpr (ADD)
#pragma unroll
                    for (int i = 0; i < 4; ++i) old[i] = fetched[i];
            }
        }
    }
    __syncthreads();
}

// Blocks: x the window (neighbours on different XCDs, a window's column blocks
// on one, so that its h comes from memory once), y the column block, z the
// halves of an adapter's rows and Z shares of the window's adapters.
//
// Bound by memory for long rows, by latency below.  Measured, us: 4096 x 11008,
// rank 64, 43 for the 180 MB of old values and results (4.2 TB/s; a copy reaches
// 4.92), with dropout 66 (masks: 2.5 times the vector instructions, two
// wavefronts to a unit; three spilled 37 registers and were a fifth slower);
// 2048 x 4096, rank 16, 10.7; 16 rows 4 to 5.  128 x 4096 of 24 adapters, rank 64,
// 14: h's 22 ranges are summed two at a time, and only then are w's loads issued.
template <int RP, bool DROP, bool ADD>
__global__ __launch_bounds__(256, RP > 64 ? 1 : 2) void expand_kernel(const Expand p) {
    __shared__ __attribute__((aligned(16))) uint16_t parts[kWindow * ExpandTile<RP>::STRIDE];
    __shared__ __attribute__((aligned(16))) float back[kWindow];
    const int lane = threadIdx.x & 63, wave = wave_of(), c16 = lane & 15, g = lane >> 4;
    const int half = p.halves > 1 ? blockIdx.z & 1 : 0, z = p.halves > 1 ? blockIdx.z >> 1 : blockIdx.z;
    const int64_t m0 = int64_t(p.window0 + int(blockIdx.x)) * kWindow;
    const int slot = slot_of(p.slots, m0 + lane, p.M, p.L);
    // the half's rows of what compact gave, at the front
    auto mine = [&](int& cnt, int& order) {
        if (p.halves == 1) return;
        order = __shfl(order, (lane + half * (kWindow / 2)) & 63);
        cnt = min(cnt - half * (kWindow / 2), kWindow / 2);
    };
    each_adapter(slot, z, p.Z, [&](int a, int cnt, int order) {
        mine(cnt, order);
        if (cnt > 0) expand_rows<RP, DROP, ADD>(p, m0, a, cnt, order, parts, back);
    });

    // rows without an adapter
    const uint64_t none = z == 0 ? __ballot(slot < 0 && m0 + lane < p.M) : 0;
    if (!none) return;
    int cnt = __builtin_popcountll(none), order = compact(none);
    mine(cnt, order);
    if (p.out && p.out != p.add)
        for (int ct = 0; ct < p.span; ++ct) {
            const int c0 = ((int(blockIdx.y) * p.span + ct) * 4 + wave) * kCols, c = held(c0 + 8 * c16, p.C);
            if (c0 >= p.C) break;
            for (int row = 0; row < cnt; row += 4) {
                const int64_t at = (m0 + __shfl(order, min(row + g, cnt - 1))) * p.C + c;
                store8(p.out + at, p.add ? load8(p.add + at) : u4{0, 0, 0, 0});
            }
        }
    if (p.sum && blockIdx.y == 0)
        for (int i0 = 0; i0 < cnt * p.R; i0 += 256) {
            const int i = i0 + threadIdx.x;
            const int64_t m = m0 + __shfl(order, (i / p.R) & 63);
            if (i < cnt * p.R) p.sum[m * p.R + i % p.R] = 0.f;
        }
}

// --------------------------------------------------------------- direct ----

struct Direct {
    const uint16_t* x;     // [M][K]
    const uint16_t* down;  // [L][R][K]
    const uint16_t* up;    // [L][R][N]
    const float* scales;
    const int32_t* slots;
    const uint16_t* base;  // [M][N], nullable, may be y
    uint16_t* y;           // [M][N]
    float* hidden;         // [M][R], nullable
    int M, R, L, K, N;
    int waves;             // wavefronts with columns of y
};

// The value of the lane N before in its row of 16, around.
template <int N>
__device__ __forceinline__ uint32_t row_rotated(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x120 + N, 0xF, 0xF, false));
}

// Both products of a decode batch in one launch, for ranks and batches up to 16.
// Blocks: x the columns, y the adapters that occur, one each.  Every block
// makes h of its adapter's rows itself, its wavefronts 512 of K's up to 4096
// channels each, in one go; the second product's operands are on their way while
// those meet, and `waves` of the wavefronts then take 128 columns each.  Bound by the
// chain of loads, with every column block reading all of an adapter's `down`: 8.2 us
// for a row of 4096 -> 4096, 10.1 for 16 rows of 16 adapters -> 12288.
template <bool ADD>
__global__ __launch_bounds__(64 * kDirectWaves) void direct_kernel(const Direct p) {
    constexpr int RP = 16, STEPS = kDirectK / (32 * kDirectWaves), COLS = 32 * STEPS;
    typedef ExpandTile<RP> T;
    __shared__ f4 sum[kDirectWaves * 64];
    __shared__ __attribute__((aligned(16))) uint16_t parts[16 * T::STRIDE];
    __shared__ __attribute__((aligned(16))) float back[16];
    const int lane = threadIdx.x & 63, wave = wave_of(), c16 = lane & 15, g = lane >> 4;
    const int y0 = (int(blockIdx.x) * p.waves + wave) * kCols, yc = held(y0 + 8 * c16, p.N);
    const bool mine = wave < p.waves && y0 < p.N;   // has columns of y
    const int slot = slot_of(p.slots, lane, p.M, p.L);

    int a = 0, cnt = 0, order = 0;   // the block's adapter and its rows
    each_adapter(slot, blockIdx.y, gridDim.y, [&](int of, int rows, int first) { a = of, cnt = rows, order = first; });
    if (cnt > 0) {
        const uint16_t* const db = p.down + int64_t(a) * p.R * p.K;
        uint32_t at[4];
        u4 raw[8], old[4], w[T::KB][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            old[i] = u4{0, 0, 0, 0};
            at[i] = uint32_t(__shfl(order, min(4 * g + i, cnt - 1))) * p.N + yc;
        }
        const uint32_t xr = uint32_t(__shfl(order, min(c16, cnt - 1))) * p.K;
        const uint32_t wr = uint32_t(min(c16, p.R - 1)) * p.K;
        f4 acc{0.f, 0.f, 0.f, 0.f};
        const int c0 = wave * COLS;
        if (c0 < p.K) {
            u4 vx[STEPS], vw[STEPS];
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int c = held(c0 + 32 * i + 8 * g, p.K);
                vx[i] = load8(off(p.x, xr + c));
                vw[i] = load8(off(db, wr + c));
            }
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                if (c0 + 32 * i >= p.K) continue;   // (K is a multiple of 32: held ones are whole steps)
                acc = mfma(vx[i], vw[i], acc);
            }
        }
        if (mine) {   // in flight while the sums meet
            load_w<RP>(raw, p.up + int64_t(a) * p.R * p.N, 0, yc, p.R, p.N);
            if constexpr (ADD)
#pragma unroll
                for (int i = 0; i < 4; ++i) old[i] = load8(off(p.base, at[i]));
        }
        sum[wave * 64 + lane] = acc;
        __syncthreads();
        if (wave == 0) {   // rows 4 g + i, column l % 16 of h, summed in order, scaled and split
            acc = sum[lane];
#pragma unroll
            for (int q = 1; q < kDirectWaves; ++q) acc += sum[q * 64 + lane];
            if (c16 >= p.R) acc = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = acc[i];   // (a bit cast of a vector's element gives its first one's)
                float inverse;
                uint32_t bits = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
                bits = bits < 0x7F800000u ? bits : 0u;   // (of the finite ones)
                bits = max(bits, row_rotated<8>(bits));
                bits = max(bits, row_rotated<4>(bits));
                bits = max(bits, row_rotated<2>(bits));
                bits = max(bits, row_rotated<1>(bits));
                const float scale = to_range(__builtin_bit_cast(float, bits), 13, inverse);
                if (c16 == 0) back[4 * g + i] = inverse;
                uint16_t* to = parts + (4 * g + i) * T::STRIDE + c16;
                uint32_t hi, lo;
                split_h(v, 0.f, scale, hi, lo);
                to[0] = uint16_t(hi);
                to[RP] = uint16_t(without_rest(hi, lo));
            }
            if (p.hidden && blockIdx.x == 0)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t m = __shfl(order, min(4 * g + i, cnt - 1));
                    if (4 * g + i < cnt && c16 < p.R) p.hidden[m * p.R + c16] = acc[i];
                }
        }
        __syncthreads();
        if (mine) {
            make_w<RP>(raw, w[0], 0, p.R);
            expand_tile<RP, false>(parts, back, w, old, p.scales[a], at, p.y, y0, yc, p.N, cnt, Drop{}, 0, 0);
        }
    }

    // rows without an adapter
    const uint64_t none = blockIdx.y == 0 ? __ballot(slot < 0 && lane < p.M) : 0;
    if (!none) return;
    cnt = __builtin_popcountll(none), order = compact(none);
    if (mine && p.y != p.base)
        for (int row = 0; row < cnt; row += 4) {
            const uint32_t at = uint32_t(__shfl(order, min(row + g, cnt - 1))) * p.N + yc;
            store8(off(p.y, at), ADD ? load8(off(p.base, at)) : u4{0, 0, 0, 0});
        }
    if (p.hidden && blockIdx.x == 0)
        for (int i0 = 0; i0 < cnt * p.R; i0 += 64 * kDirectWaves) {
            const int i = i0 + threadIdx.x;
            const int64_t m = __shfl(order, (i / p.R) & 63);
            if (i < cnt * p.R) p.hidden[m * p.R + i % p.R] = 0.f;
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
    int C, tiles;          // tiles of 128 columns
};
struct Outer {
    OuterJob job[2];
    const float* scales;
    const int32_t* start;  // [L + 1], null: adapter 0 takes every row
    const int32_t* list;
    int M, R, L, splits, rchunks;
    int adapter0;          // of this launch
};

// Rows of one adapter against 128 columns and 16 RW of the rank.  The block's
// four wavefronts take 32 rows each, a matrix step: src through dropout into
// fragments, h into fragments of its 16s.  The products of a step go to RW
// wavefronts, 16 of the rank each, over LDS (RW = 1: to itself).  So the rows
// are read, masked and split once whatever the rank, and a wavefront's sums
// take 32 registers.  With RW < 4 groups of RW wavefronts take different rows
// and meet at the end.  The next rows' loads are in flight during the products.
//
// h is split in two fp16 numbers after a power of two for each step and column
// has brought it into their range; the step's products are brought back as they
// are added to the fp32 sums.
// Blocks: x the column tiles of both gradients, y the range of rows, z the
// rank's 64s and the adapter.
//
// Bound by vector instructions: masks (half of them, with dropout), the split of
// h, addresses; then by latency.  Measured, us: 4096 rows of 4 adapters, C = 11008
// and 4096, rank 64, dropout, 73 to 76 for the 124 MB read (every 16 of the rank
// masking for itself: 81 to 92); 2048 rows, C = 4096 twice, rank 16, 12.3 to 13.0
// in 16 ranges of a single round each, whose rows are loaded twice.
template <int RW, bool LIST>
__global__ __launch_bounds__(256, 2) void outer_kernel(const Outer p) {
    __shared__ u4 xs[4 * 8 * 64];                        // [step][column fragment][lane]
    __shared__ u4 hs[RW > 1 ? 4 * RW * 2 * 64 : 1];      // [step][16 of the rank][first, second part][lane]
    __shared__ f4 back[RW > 1 ? 4 * RW * 4 : 1];         // [step][16 of the rank][16]: the powers' inverses
    const int lane = threadIdx.x & 63, wave = wave_of(), c16 = lane & 15, g = lane >> 4;
    const int group = wave / RW * RW;   // the first wavefront whose rows this one takes
    const int mine = wave - group;      // which 16 of the rank: r0 + RW * (row of the fragment) + mine
    const bool second = int(blockIdx.x) >= p.job[0].tiles;
    const OuterJob& j = p.job[second];
    const int tile = blockIdx.x - (second ? p.job[0].tiles : 0), split = blockIdx.y;
    const int r0 = p.rchunks > 1 ? (blockIdx.z & 1) * 64 : 0;
    const int a = p.adapter0 + int(p.rchunks > 1 ? blockIdx.z >> 1 : blockIdx.z);
    const int at = LIST ? p.start[a] : 0, cnt = LIST ? p.start[a + 1] - at : a == 0 ? p.M : 0;
    const int c = held(tile * kCols + 8 * c16, j.C);
    const bool drop = j.drop.t != 0;
    const uint64_t stream = drop ? wq::drop_stream(j.drop) : 0;
    // rounds of four steps of 32 rows
    const int rounds = (cnt + 127) / 128, end = int(int64_t(split + 1) * rounds / p.splits);
    const int begin = int(int64_t(split) * rounds / p.splits);
    // a lane's r: RW side by side; past the rank others are taken, and what they give is not kept
    const int held_r = min(r0 + RW * c16, p.R - RW);
    f4 acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = f4{0.f, 0.f, 0.f, 0.f};

    // Rows 8 g + i of the wavefront's step.  Past the adapter's: the list's next
    // ones, which exist, or the last one.  (No branch joins behind these loads: the
    // wait for them would be one for the products' loads before them.)
    auto rows = [&](int of, int (&m)[8]) {
        const int n = of * 128 + wave * 32 + 8 * g;
        if constexpr (LIST)
            __builtin_memcpy(m, p.list + at + n, 32);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = min(n + i, p.M - 1);
    };
    typedef float hvec __attribute__((ext_vector_type(RW)));
    u4 x[8];
    hvec hv[8];
    int m[8], next[8];
    auto load = [&] {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = load8(j.src + int64_t(m[i]) * j.C + c);
            __builtin_memcpy(&hv[i], j.h + int64_t(m[i]) * p.R + held_r, 4 * RW);
        }
    };
    if (begin < end) {
        rows(begin, m);
        load();
        rows(min(begin + 1, end - 1), next);
    }
#pragma unroll 1
    for (int round = begin; round < end; ++round) {
        const int first = round * 128 + wave * 32 + 8 * g;   // the lane's first row in the adapter's
        float h[8][RW];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int t = 0; t < RW; ++t) h[i][t] = hv[i][t];
        if (drop)
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                uint64_t n[4];
                u4 keep[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) n[k] = (uint64_t(m[i + k]) * j.C + c) >> 3;
                wq::keep8(n, j.drop, stream, keep);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[i + k] &= keep[k];
            }
        if (RW > 1 && p.R % RW) {   // a lane whose r's end inside RW of them took the rank's last RW
            const int by = r0 + RW * c16 - held_r;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v[RW];
#pragma unroll
                for (int t = 0; t < RW; ++t) {
                    v[t] = h[i][t];
#pragma unroll
                    for (int k = 1; t + k < RW; ++k) v[t] = by == k ? h[i][t + k] : v[t];
                }
#pragma unroll
                for (int t = 0; t < RW; ++t) h[i][t] = v[t];
            }
        }
        if (round * 128 + 128 > cnt)   // rows past the adapter's count as zeros
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (first + i >= cnt) {
                    x[i] = u4{0, 0, 0, 0};
#pragma unroll
                    for (int t = 0; t < RW; ++t) h[i][t] = 0.f;
                }
        u4 w[8], hi[RW], lo[RW];
        f4 own{0.f, 0.f, 0.f, 0.f};   // RW = 1: the wavefront's inverses
        transpose8(x, w);
#pragma unroll
        for (int t = 0; t < RW; ++t) {
            float all[8], inverse;
#pragma unroll
            for (int i = 0; i < 8; ++i) all[i] = h[i][t];
            bool odd;
            float most = largest(all, odd);
            most = __builtin_fmaxf(most, __shfl_xor(most, 16));
            most = __builtin_fmaxf(most, __shfl_xor(most, 32));
            const float scale = to_range(most, 13, inverse);
            if (RW == 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) own[i] = __shfl(inverse, 4 * g + i);
            else if (g == 0)
                reinterpret_cast<float*>(back)[(wave * RW + t) * 16 + c16] = inverse;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t u, v;
                split_h(all[2 * i], all[2 * i + 1], scale, u, v);
                hi[t][i] = u;
                lo[t][i] = v;
            }
            if (odd)
#pragma unroll
                for (int i = 0; i < 4; ++i) lo[t][i] = without_rest(hi[t][i], lo[t][i]);
        }
        if constexpr (RW > 1) {
#pragma unroll
            for (int k = 0; k < 8; ++k) xs[(wave * 8 + k) * 64 + lane] = w[k];
#pragma unroll
            for (int t = 0; t < RW; ++t) {
                hs[((wave * RW + t) * 2 + 0) * 64 + lane] = hi[t];
                hs[((wave * RW + t) * 2 + 1) * 64 + lane] = lo[t];
            }
        }
        // (the last round loads its own rows again: a branch would end in a wait for them)
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = next[i];
        load();
        rows(min(round + 2, end - 1), next);
        if (RW > 1) __syncthreads();
#pragma unroll
        for (int q = 0; q < RW; ++q) {
            const int step = group + q;
            const u4 vh = RW > 1 ? hs[((step * RW + mine) * 2 + 0) * 64 + lane] : hi[0];
            const u4 vl = RW > 1 ? hs[((step * RW + mine) * 2 + 1) * 64 + lane] : lo[0];
            const f4 f = RW > 1 ? back[(step * RW + mine) * 4 + g] : own;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const u4 v = RW > 1 ? xs[(step * 8 + k) * 64 + lane] : w[k];
                f4 t{0.f, 0.f, 0.f, 0.f};
                t = mfma(vh, v, t);
                t = mfma(vl, v, t);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[k][i] = __builtin_fmaf(t[i], f[i], acc[k][i]);
            }
        }
        if (RW > 1) __syncthreads();
    }

    if constexpr (RW < 4) {   // the wavefronts of different rows, in order
        f4* const sums = reinterpret_cast<f4*>(xs);
        if (group)
#pragma unroll
            for (int k = 0; k < 8; ++k) sums[(wave * 8 + k) * 64 + lane] = acc[k];
        __syncthreads();
        if (group) return;
#pragma unroll
        for (int o = RW; o < 4; o += RW)
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] += sums[((wave + o) * 8 + k) * 64 + lane];
    }

    if (any_odd(acc)) {   // row by row in fp32, the loads of four at once
        f4 plain[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) plain[k] = f4{0.f, 0.f, 0.f, 0.f};
        const int last = int(std::min(int64_t(end) * 128, int64_t(cnt)));
#pragma unroll 1
        for (int n = begin * 128; n < last; n += 4) {
            u4 v[4], keep[4];
            f4 q[4];
            uint64_t eight[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int nth = min(n + u, last - 1);
                const int64_t row = LIST ? p.list[at + nth] : nth;
                eight[u] = (uint64_t(row) * j.C + c) >> 3;
                v[u] = load8(j.src + row * j.C + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) q[u][i] = j.h[row * p.R + min(r0 + RW * (4 * g + i) + mine, p.R - 1)];
            }
            if (drop) {
                wq::keep8(eight, j.drop, stream, keep);
#pragma unroll
                for (int u = 0; u < 4; ++u) v[u] &= keep[u];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (n + u >= last) break;
                float f[8];
                wq::load_h<8>(reinterpret_cast<const uint16_t*>(&v[u]), f);
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) plain[k][i] = __builtin_fmaf(q[u][i], f[k], plain[k][i]);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[k][i] = finite(acc[k][i]) ? acc[k][i] : plain[k][i];
    }

    const float s = (drop ? j.drop.keep : 1.f) * (cnt ? p.scales[a] : 0.f);
    float* to = (p.splits > 1 ? j.part + int64_t(split) * p.L * p.R * j.C : j.dw) + int64_t(a) * p.R * j.C + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + RW * (4 * g + i) + mine;
        if (r >= p.R) continue;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = acc[k][i] * s;
        __builtin_memcpy(to + int64_t(r) * j.C, v, 32);
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
    f4 v{0.f, 0.f, 0.f, 0.f};
    if (size - q >= 4) {
        const float* at = j.part + q;
#pragma unroll 8
        for (int s = 0; s < p.splits; ++s, at += size) {
            f4 w;
            __builtin_memcpy(&w, at, 16);
            v += w;
        }
        __builtin_memcpy(j.dw + q, &v, 16);
        return;
    }
    for (int64_t i = q; i < size; ++i) {
        float w = 0.f;
        for (int s = 0; s < p.splits; ++s) w += j.part[s * size + i];
        j.dw[i] = w;
    }
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
__global__ __launch_bounds__(64 * kShrinkWaves) void list_kernel(const Shrink p) {
    __shared__ int counts[2 * kShrinkWaves];
    list_rows(p, int(blockIdx.x), counts);
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

template <int N>
using Int = std::integral_constant<int, N>;

// launch(now, first) for 0 .. total - 1, at most `most` at a time.
template <class Launch>
wq_status pieces(int64_t total, int64_t most, const Launch& launch) {
    for (int64_t first = 0; first < total; first += most) {
        launch(unsigned(std::min(total - first, most)), first);
        const wq_status st = wqh::launch_status();
        if (st != WQ_OK) return st;
    }
    return WQ_OK;
}
constexpr int kMaxY = 65535;        // blocks of a launch in y or z
constexpr int kMaxWidth = 1 << 22;  // adapters, and columns

// How many blocks share the work of a window whose adapters are not known here,
// where `blocks` alone leave units idle.
int shares(int M, int L, int64_t blocks, int want) {
    return int(std::max<int64_t>(1, std::min<int64_t>(std::min(std::min(L, M), kWindow), want / blocks)));
}

// Batches of fewer than 16 rows to an adapter are taken for decode batches: the
// shrink takes 16 rows at a time (us against 64 at a time, the whole call, K = N
// = 4096, rank 16: 128 rows of 32 adapters 10.7 and 16.9, 1000 rows of 100 in any
// order 59 and 123, in runs 16.5 and 26.0; above the border, 256 rows of 8 in
// runs, 10.3 and 9.8, 200 rows of 4 at rank 64, 23.3 and 14.9).
bool mixed(const int32_t* slots, int M, int L) { return slots && M < 16LL * L; }

// Ranges of the long side of a shrink, and the blocks that share a window: one
// round of blocks on 256 units (two took 55.7 us instead of 47.8 for a whole call
// of 4096 rows, K = 4096, N = 11008, rank 64: every range is read again by the
// second product).
struct ShrinkPlan {
    int splits, cps, Z;
    ShrinkPlan(int M, int R, int L, int C) {
        const int chunks = div_up(C, kChunk), rchunks = padded_rank(R) > 64 ? 2 : 1;
        const int64_t base = int64_t(div_up(M, kWindow)) * rchunks;
        const int want = int(std::min<int64_t>(std::max<int64_t>(256 / base, 1), 32));
        cps = div_up(chunks, std::min(want, div_up(chunks, 4)));
        splits = div_up(chunks, cps);
        Z = shares(M, L, base * splits, M < 16LL * L ? 512 : 256);
    }
    size_t bytes(int M, int R) const { return round256(size_t(splits) * M * padded_rank(R) * 4); }
};

wq_status shrink(const wqh::Adapters& a, const uint16_t* src, const uint16_t* w, const Drop& d, float* part, int C,
                 int32_t* start, int32_t* list, hipStream_t s) {
    const ShrinkPlan plan(a.M, a.R, a.L, C);
    const int RP = padded_rank(a.R);
    Shrink p{src, w, a.slots, part, d, a.M, a.R, a.L, C, plan.splits, plan.cps, plan.Z, RP > 64 ? 2 : 1, start, list, 0, 0};
    const int lists = start ? a.L : 0;   // blocks
    constexpr int T = 64 * kShrinkWaves;
    auto list_all = [&] {
        return pieces(lists, kMaxWidth, [&](unsigned now, int64_t) { list_kernel<<<now, T, 0, s>>>(p); });
    };
    if (C < 8) {   // (N: K is 32 at least, so nothing is dropped)
        const wq_status st = pieces((int64_t(a.M) * RP + 255) / 256, wqh::kMaxBlocks, [&](unsigned now, int64_t first) {
            narrow_shrink_kernel<<<now, 256, 0, s>>>(p, RP, first);
        });
        return st != WQ_OK ? st : list_all();
    }
    const bool one = a.M <= 16 || mixed(a.slots, a.M, a.L);
    const unsigned zs = unsigned(p.Z * p.rchunks);
    int layers = div_up(lists, int64_t(p.splits) * zs);
    if (layers > 16) {   // a launch of their own
        layers = 0;
        const wq_status st = list_all();
        if (st != WQ_OK) return st;
    }
    return pieces(div_up(a.M, kWindow), kMaxY - 16, [&](unsigned windows, int64_t first) {
        p.window0 = int(first);
        p.lists = first == 0 ? layers : 0;
        const dim3 grid(unsigned(p.splits), unsigned(p.lists) + windows, zs);
        auto go = [&](auto n) {
            constexpr int NRT = decltype(n)::value;
            if (one && !d.t)
                shrink_kernel<NRT, false, true><<<grid, T, 0, s>>>(p);
            else if (one)
                shrink_kernel<NRT, true, true><<<grid, T, 0, s>>>(p);
            else if (!d.t)
                shrink_kernel<NRT, false, false><<<grid, T, 0, s>>>(p);
            else
                shrink_kernel<NRT, true, false><<<grid, T, 0, s>>>(p);
        };
        if (RP == 16)
            go(Int<1>{});
        else if (RP == 32)
            go(Int<2>{});
        else
            go(Int<4>{});
    });
}

wq_status expand(const wqh::Adapters& a, const float* part, int splits, const uint16_t* w, const Drop& d,
                 const uint16_t* add, uint16_t* out, float* sum, int C, hipStream_t s) {
    Expand p{part, w, a.scales, a.slots, add, out, sum, d, a.M, a.R, a.L, C, splits, 1, 1, 1, 0};
    if (out && C < 8)
        return pieces((int64_t(a.M) * C + 255) / 256, wqh::kMaxBlocks, [&](unsigned now, int64_t first) {
            narrow_expand_kernel<<<now, 256, 0, s>>>(p, padded_rank(a.R), first);
        });
    const int64_t windows = div_up(a.M, kWindow);
    const int wide = out ? div_up(C, 4 * kCols) : 1;   // blocks of 512 columns
    // columns to a block so that two blocks to a unit run in one round (4096 x
    // 11008, rank 64: 42.8 us, with dropout 66.9; 512 to a block, 2.75 rounds, 46.0
    // and 72.2)
    p.span = int(std::max<int64_t>(1, std::min<int64_t>(std::min(wide, 8), (windows * wide + 511) / 512)));
    const int cblocks = div_up(wide, p.span);
    // (2048 rows, K = N = 4096, rank 16: 14.8 us with halves, 15.5 without)
    p.halves = a.M > kWindow / 2 && !mixed(a.slots, a.M, a.L) && windows * cblocks < 512 ? 2 : 1;
    p.Z = shares(a.M, a.L, windows * cblocks * p.halves, 512);
    return pieces(windows, wqh::kMaxBlocks, [&](unsigned now, int64_t first) {
        p.window0 = int(first);
        const dim3 grid(now, unsigned(cblocks), unsigned(p.Z * p.halves));
        auto go = [&](auto n) {
            constexpr int RP = decltype(n)::value;
            if (d.t && add)
                expand_kernel<RP, true, true><<<grid, 256, 0, s>>>(p);
            else if (d.t)
                expand_kernel<RP, true, false><<<grid, 256, 0, s>>>(p);
            else if (add)
                expand_kernel<RP, false, true><<<grid, 256, 0, s>>>(p);
            else
                expand_kernel<RP, false, false><<<grid, 256, 0, s>>>(p);
        };
        switch (padded_rank(a.R)) {
            case 16: go(Int<16>{}); break;
            case 32: go(Int<32>{}); break;
            case 64: go(Int<64>{}); break;
            default: go(Int<128>{});
        }
    });
}

// Whether a forward pass without dropout is one launch.  It saves a caller who
// launches from the host 4.5 of 14.2 us, a launch and a workspace.  On the GPU itself,
// in a replayed graph, it gains for short rows and loses at the longest (us, one
// launch and two; rank 16: K = N = 1024, 1 row 4.4 and 6.2, 16 rows of 16 adapters
// 5.1 and 8.1; K = 2048, N = 11008, rank 8, 16 of 16 6.3 and 8.4; K = N = 4096, 1 row
// 7.6 and 6.6, 4 of one adapter 8.9 and 7.1, 16 of 16 9.2 and 8.3): one block reads an
// adapter's whole `down`.  Many rows of one adapter (16: 10.8 and 7.6), wider ranks
// (32, 8 rows: 12.4 and 8.5) and longer rows (K = 11008: 21.7 and 12.2) lost more than
// the launch saves, measured before the form was held to a block's registers.
bool direct_fits(int M, int N, int K, int R, int L) {
    return M <= kDirectM && M <= 4LL * L && R <= 16 && K <= kDirectK && N >= 8;
}

wq_status direct(const wqh::Adapters& a, const uint16_t* x, const uint16_t* down, const uint16_t* up,
                 const uint16_t* base, uint16_t* y, float* hidden, int N, int K, hipStream_t s) {
    Direct p{x, down, up, a.scales, a.slots, base, y, hidden, a.M, a.R, a.L, K, N, 4};
    const int Z = std::min(a.L, a.M);   // adapters that can occur
    if (int64_t(div_up(N, 4 * kCols)) * Z > 256) p.waves = kDirectWaves;
    const dim3 grid(unsigned(div_up(N, p.waves * kCols)), unsigned(Z));
    if (base)
        direct_kernel<true><<<grid, 64 * kDirectWaves, 0, s>>>(p);
    else
        direct_kernel<false><<<grid, 64 * kDirectWaves, 0, s>>>(p);
    return wqh::launch_status();
}

// Ranges of rows of the gradients: about four blocks to a unit, as blocks with
// dropout's masks and without are of unequal length (4096 rows of 4 adapters, K =
// 11008, N = 4096, rank 64: 82 us with two ranges and their sum, 112 with one),
// and no more than an adapter's share of the rows fills.
int outer_splits(int M, int R, int L, int K, int N) {
    const int64_t blocks = int64_t(L) * (padded_rank(R) > 64 ? 2 : 1) * (div_up(K, kCols) + div_up(N, kCols));
    return int(std::max<int64_t>(1, std::min<int64_t>(std::min(div_up(div_up(M, L), 128), 32), 1024 / blocks)));
}

wq_status outer(const wqh::Adapters& a, Outer& p, hipStream_t s) {
    const int RP = padded_rank(a.R);
    p.rchunks = RP > 64 ? 2 : 1;
    const bool narrow = p.job[1].C < 8;
    for (OuterJob& j : p.job) j.tiles = div_up(j.C, kCols);
    if (narrow) {
        const wq_status st = pieces(int64_t(a.L) * a.R * p.job[1].C, wqh::kMaxBlocks, [&](unsigned now, int64_t first) {
            narrow_outer_kernel<<<now, 64, 0, s>>>(p, first);
        });
        if (st != WQ_OK) return st;
    }
    const unsigned tiles = unsigned(p.job[0].tiles + (narrow ? 0 : p.job[1].tiles));
    wq_status st = pieces(a.L, kMaxY / 2, [&](unsigned now, int64_t first) {
        p.adapter0 = int(first);
        const dim3 grid(tiles, unsigned(p.splits), now * unsigned(p.rchunks));
        auto go = [&](auto rw) {
            if (p.list)
                outer_kernel<decltype(rw)::value, true><<<grid, 256, 0, s>>>(p);
            else
                outer_kernel<decltype(rw)::value, false><<<grid, 256, 0, s>>>(p);
        };
        if (RP == 16)
            go(Int<1>{});
        else if (RP == 32)
            go(Int<2>{});
        else
            go(Int<4>{});
    });
    if (st != WQ_OK || p.splits == 1) return st;
    const int64_t n0 = (int64_t(a.L) * a.R * p.job[0].C + 3) / 4 * 4;
    const int64_t n1 = narrow ? 0 : int64_t(a.L) * a.R * p.job[1].C;
    return pieces((n0 + n1 + 1023) / 1024, wqh::kMaxBlocks, [&](unsigned now, int64_t first) {
        outer_sum_kernel<<<now, 256, 0, s>>>(p, n0, first * 256);
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
        list = take((size_t(M) + kPad) * 4);
        outer0 = take(grads * K);
        outer1 = take(grads * N);
        bytes = at;
    }
};

}  // namespace

namespace wqh {

size_t adapters_workspace(int M, int N, int K, int R, int L, bool dropping) {
    return !dropping && direct_fits(M, N, K, R, L) ? 0 : ShrinkPlan(M, R, L, K).bytes(M, R);
}

wq_status adapters_forward(const Adapters& a, const uint16_t* x, const uint16_t* down, const uint16_t* up,
                           const uint16_t* base, uint16_t* y, float* hidden, int N, int K, void* ws, hipStream_t s) {
    if (!a.drop.t && direct_fits(a.M, N, K, a.R, a.L)) return direct(a, x, down, up, base, y, hidden, N, K, s);
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
