// Shared parts of the feed-forward block's kernels (wq_block.h): activations
// and their derivatives, the forward epilogue, fp16 vector accesses.
#pragma once

#include <algorithm>

#include "../../include/wq_block.h"
#include "wq_gemm_common.h"

namespace wq {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float h2f(uint16_t v) { return float(__builtin_bit_cast(_Float16, v)); }
__device__ __forceinline__ uint16_t f2h(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

// Items (of `total`, spread evenly over steps first .. first + len - 1) that
// fall on step m.
constexpr int step_share(int total, int first, int len, int m) {
    return m < first || m >= first + len ? 0 : total * (m - first + 1) / len - total * (m - first) / len;
}

// Issue order of one k-step of a software-pipelined product: after each of
// its NM matrix instructions a share of the step's NR LDS reads (first half),
// NS LDS writes and NL loads (second half), and NV vector instructions.  In-order
// issue would otherwise hold all of them behind the matrix instructions.
template <int NM, int NR, int NS, int NL, int NV, int M = 0>
__device__ __forceinline__ void sched_step() {
    if constexpr (M < NM) {
        constexpr int H = NM / 2;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr (step_share(NR, 0, H, M) > 0)
            __builtin_amdgcn_sched_group_barrier(0x100, step_share(NR, 0, H, M), 0);
        if constexpr (step_share(NS, H, NM - H, M) > 0)
            __builtin_amdgcn_sched_group_barrier(0x200, step_share(NS, H, NM - H, M), 0);
        if constexpr (step_share(NL, H, NM - H, M) > 0)
            __builtin_amdgcn_sched_group_barrier(0x020, step_share(NL, H, NM - H, M), 0);
        __builtin_amdgcn_sched_group_barrier(0x002, NV, 0);
        sched_step<NM, NR, NS, NL, NV, M + 1>();
    } else {
        __builtin_amdgcn_sched_barrier(0);
    }
}

// What a tile kernel's block does under a TilePlan: its tile's coordinates,
// whether its product is partial, and which partial product it is.
struct TileWork {
    int m_t, n_t, split;
    long long part;  // (split, tile of the tail), -1 for a whole tile
};

// Tile t of m_tiles x n_tiles: consecutive tiles cover strips of four M-tiles,
// so that what runs at a time is a compact rectangle.
__device__ __forceinline__ void tile_place(int t, int m_tiles, int n_tiles, int& m_t, int& n_t) {
    constexpr int GM = 4;
    const int group = t / (GM * n_tiles), first_m = group * GM;
    const int gsm = min(m_tiles - first_m, GM), r = t - group * (GM * n_tiles);
    m_t = first_m + r % gsm;
    n_t = r / gsm;
}

// Blocks are dealt to the XCDs round-robin; each gets contiguous tiles.
__device__ __forceinline__ TileWork tile_work(int b, int tiles, int head, int m_tiles, int n_tiles) {
    TileWork w;
    int t;
    if (b < head) {
        t = xcd_tile(b, head, 8);
        w.split = 0;
        w.part = -1;
    } else {
        const int tail = tiles - head, q = b - head;
        w.split = q / tail;
        const int i = xcd_tile(q - w.split * tail, tail, 8);
        t = head + i;
        w.part = (long long)w.split * tail + i;
    }
    tile_place(t, m_tiles, n_tiles, w.m_t, w.n_t);
    return w;
}

// ------------------------------------------------ copies into LDS ----
//
// Tiles go from memory straight into LDS (no registers, no LDS writes, which
// hold a wavefront up by 25 cycles each where a read costs it 3).  A copy is
// an asm statement that writes no register: for its own form the compiler
// would wait for every copy in flight before any read of LDS that it cannot
// tell from the copy's target.  It does not know of these copies, so
//  - a target must be free when the copy is issued: behind the barrier that
//    follows its last reads;
//  - copies_landed<N>() (all but the wavefront's newest N loads and copies
//    are complete) comes before the barrier that publishes them;
//  - a kernel that leaves copies in flight across its waits (N > 0) has no
//    other memory loads there, or waits for them too.
// m0, the target's LDS address, is an operand: the compiler sets it and keeps
// its own uses of it apart.

// Buffer resource over `bytes` bytes at p (at most 2 GiB of them): accesses
// add a 32-bit offset to it, and those past its end read zeros.
__device__ __forceinline__ u4 copy_source(const void* p, uint64_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    u4 r;
    r.x = __builtin_amdgcn_readfirstlane(uint32_t(at));
    r.y = __builtin_amdgcn_readfirstlane(uint32_t(at >> 32) & 0xFFFFu);  // stride 0
    r.z = __builtin_amdgcn_readfirstlane(bytes < 0x80000000u ? uint32_t(bytes) : 0x80000000u);
    r.w = 0x00020000u;  // raw 32-bit data
    return r;
}
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every resource's end

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return uint32_t(reinterpret_cast<uintptr_t>((lptr_t)(p)));
}

// Lane l's B bytes at offset `off` to lds + 16 l (B = 16 and 12) or lds + 4 l
// (2 and 1, zero-extended to 4 bytes).
template <int B>
__device__ __forceinline__ void copy_to_lds(u4 src, uint32_t off, uint32_t lds) {
    const uint32_t l = __builtin_amdgcn_readfirstlane(lds);
    if constexpr (B == 16)
        asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "{m0}"(l), "v"(off), "s"(src));
    else if constexpr (B == 12)
        asm volatile("s_nop 0\n\tbuffer_load_dwordx3 %1, %2, 0 offen lds" : : "{m0}"(l), "v"(off), "s"(src));
    else if constexpr (B == 2)
        asm volatile("s_nop 0\n\tbuffer_load_ushort %1, %2, 0 offen lds" : : "{m0}"(l), "v"(off), "s"(src));
    else
        asm volatile("s_nop 0\n\tbuffer_load_ubyte %1, %2, 0 offen lds" : : "{m0}"(l), "v"(off), "s"(src));
}

template <int N>
__device__ __forceinline__ void copies_landed() {
    static_assert(N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// 64-column stages of a BM-row tile of a row-major fp16 matrix, into
// [BM][64] with 16-byte unit u of row r at position u ^ ((r / 2) mod 8): 16
// consecutive rows read at one u fall on all 64 banks.  Copy i of a wavefront
// fills rows 8 (wave COPIES + i) + l / 8, lane l the row's position l % 8;
// eight lanes read one 128-byte line.  Rows past the matrix and columns past
// `cols` (a multiple of 8) become zeros.  Offsets are below 2^31: 256 rows of
// at most 2^22 columns.
template <int BM>
struct TileCopy {
    static constexpr int COPIES = BM / 32;  // of 1 KB per wavefront and stage
    u4 src;
    uint32_t off[2];  // byte offset of an even and of an odd copy, without its 8-row steps
    uint32_t u0;      // unit of an even copy (an odd one's is u0 ^ 4)
    uint32_t cols, row8, wave;

    // first: the tile's first row; rows: how many the matrix has from there
    __device__ __forceinline__ TileCopy(const uint16_t* first, int rows, int cols_, int wave_, int lane)
        : src(copy_source(first, uint64_t(uint32_t(rows)) * uint32_t(cols_) * 2u)), cols(cols_),
          row8(uint32_t(cols_) * 16u), wave(wave_) {
        u0 = uint32_t(lane & 7) ^ uint32_t(lane >> 4);  // (row / 2) % 8 of an even copy: l / 16
#pragma unroll
        for (int e = 0; e < 2; ++e)
            off[e] = (uint32_t(lane >> 3) + 8u * (wave * COPIES + e)) * cols * 2u + unit(e) * 16u;
    }
    __device__ __forceinline__ uint32_t unit(int e) const { return u0 ^ (e ? 4u : 0u); }
    // Where a stage's even and odd copies read, and their first target.
    struct Stage {
        uint32_t off[2], lds;
    };
    __device__ __forceinline__ Stage stage(int st, const uint8_t* buf) const {
        Stage s;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            s.off[e] = uint32_t(st) * 64u + 8u * unit(e) < cols ? off[e] + uint32_t(st) * 128u : kNowhere;
        s.lds = lds_address(buf) + wave * COPIES * 1024u;
        return s;
    }
    __device__ __forceinline__ void copy(const Stage& s, int i) const {
        copy_to_lds<16>(src, s.off[i & 1] + uint32_t(i >> 1) * 2u * row8, s.lds + uint32_t(i) * 1024u);
    }
    __device__ __forceinline__ void copy(const Stage& s, int i0, int i1) const {
#pragma unroll
        for (int i = i0; i < i1; ++i) copy(s, i);
    }
};

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

// act(v) and act'(v).  v is held within +-100 for the derivative (it is 0 or 1
// there to fp32's accuracy, and so is the factor that both share).
__device__ __forceinline__ float act_slope(float v, int kind, float& value) {
    const float low = v < -100.f ? -100.f : v, c = low > 100.f ? 100.f : low;
    switch (kind) {
        case WQ_ACT_RELU:
            value = v < 0.f ? 0.f : v;
            return v > 0.f ? 1.f : v != v ? v : 0.f;
        case WQ_ACT_GELU: {
            const float t = 0.5f * erfcf(-kSqrtHalf * c);
            value = low * t;
            return __builtin_fmaf(c * kInvSqrt2Pi, __expf(-0.5f * c * c), t);
        }
        case WQ_ACT_GELU_TANH: {
            const float t = sigmoid(2.f * kTanhScale * __builtin_fmaf(kTanhCubic * c * c, c, c));
            const float du = 2.f * kTanhScale * __builtin_fmaf(3.f * kTanhCubic * c, c, 1.f);
            value = low * t;
            return __builtin_fmaf(c * t * (1.f - t), du, t);
        }
        case WQ_ACT_SILU: {
            const float t = sigmoid(c);
            value = low * t;
            return t * __builtin_fmaf(c, 1.f - t, 1.f);
        }
        default: value = v; return 1.f;
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

// Sums over `splits` partial products, `step` floats apart, of four
// neighbouring columns per entry of `at` (multiples of 4), in order; up to four
// products' loads are in flight at once.
template <int P>
__device__ __forceinline__ void sum_ranges(const float* __restrict__ src, const int (&at)[P], size_t step, int splits,
                                           f4 (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = f4{0.f, 0.f, 0.f, 0.f};
    auto add = [&](auto n) {
        f4 w[decltype(n)::value][P];
#pragma unroll
        for (int s = 0; s < decltype(n)::value; ++s)
#pragma unroll
            for (int i = 0; i < P; ++i) w[s][i] = *reinterpret_cast<const f4*>(src + s * step + at[i]);
#pragma unroll
        for (int s = 0; s < decltype(n)::value; ++s)
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] += w[s][i];
        src += decltype(n)::value * step;
    };
    int s = splits;
    for (; s >= 4; s -= 4) add(std::integral_constant<int, 4>{});
    if (s >= 2) add(std::integral_constant<int, 2>{});
    if (s & 1) add(std::integral_constant<int, 1>{});
}

}  // namespace wq

namespace wqh {

// A launch holds fewer than 2^32 threads in x: blocks of 256 threads.
constexpr long long kMaxBlocks = (1LL << 24) - 1;

// launch(blocks, first) for blocks 0 .. total - 1 (total below 2^31), in as
// many launches as that takes.
template <class Launch>
wq_status launch_pieces(long long total, const Launch& launch) {
    for (long long first = 0; first < total; first += kMaxBlocks) {
        launch(unsigned(std::min(total - first, kMaxBlocks)), int(first));
        const wq_status st = launch_status();
        if (st != WQ_OK) return st;
    }
    return WQ_OK;
}

// Time of a tile kernel's block, in us on MI355X: `idle` + `load` * (share of
// the compute units that work) per 64-deep stage, plus `fixed` per tile (the
// clock falls as more units feed their matrix cores).  `overlap`: two blocks
// share a unit, so that rounds need not be whole.
struct TileCost {
    int BM;
    double idle, load, fixed;
    bool overlap;
};
// A tile kernel's heights, and what cutting tiles adds: `cut` us for the second
// kernel and `cut_mb` for each MB (10^6 bytes) of partial products.
struct TileCosts {
    TileCost height[3];
    double cut, cut_mb;
};
// How a tile kernel covers its tiles: tiles 0 .. head - 1 whole, the others cut
// into `splits` ranges of `sps` stages, whose fp32 partial products meet in a
// second kernel.
struct TilePlan {
    int BM = 128, splits = 1, sps = 0, tiles = 0, head = 0;
    int tail() const { return tiles - head; }
    unsigned blocks() const { return unsigned(head) + unsigned(tail()) * unsigned(splits); }
    size_t part_bytes() const { return size_t(tail()) * splits * BM * 256 * 4; }
};

// Tile height and cut with the least modelled time: blocks run in rounds of
// one per unit; whole rounds run whole, and what a last, partly filled round
// would hold may be cut (or everything, when there is less than a round).  A
// cut writes and re-reads its partial products and launches a second kernel.
// Ranges are multiples of `align` stages, at least four.  The costs are fitted
// to 6723 timings of the two tile kernels (M = 33 .. 2048, five layers from
// 1024 x 2048 to 4096 x 11008, three widths and group sizes, all heights, 1 ..
// 32 ranges, with and without whole rounds): over each kernel's timings the
// choice is 0.3 .. 2.2 % slower than the fastest on average, 17 % at worst.
// all_part: every product goes through the second kernel.  No tiles: what
// has to be cut does not fit part_bytes, or no height fits a launch.
inline TilePlan plan_tiles(int M, int n_tiles, int stages, const TileCosts& costs, int align, size_t part_bytes,
                           int units, bool all_part) {
    TilePlan best;
    double best_us = 1e300;
    for (const TileCost& c : costs.height) {
        const long long tiles_ll = (long long)((M + c.BM - 1) / c.BM) * n_tiles;
        if (tiles_ll > kMaxBlocks) continue;
        const int tiles = int(tiles_ll);
        auto round_us = [&](int st, double share) { return st * (c.idle + c.load * share) + c.fixed; };
        // `blocks` of st stages in rounds
        auto run_us = [&](double blocks, int st) {
            if (blocks <= units) return blocks > 0 ? round_us(st, blocks / units) : 0.0;
            if (c.overlap) return round_us(st, 1.0) * (blocks / units);
            const double whole = double((long long)(blocks / units)), rest = blocks / units - whole;
            return whole * round_us(st, 1.0) + (rest > 0 ? round_us(st, rest) : 0.0);
        };
        const int whole = tiles / units * units;
        for (int pass = 0; pass < 2; ++pass) {
            const int head = pass == 0 ? 0 : whole;
            if (pass == 1 && (head == 0 || head == tiles || all_part)) continue;
            for (int S = 1; S <= 32; ++S) {
                const int sps = ((stages + S - 1) / S + align - 1) / align * align;
                if ((stages + sps - 1) / sps != S || (S == 1 && pass == 1)) continue;
                TilePlan p{c.BM, S, sps, tiles, S == 1 && !all_part ? tiles : head};
                if (p.head + (long long)p.tail() * S > kMaxBlocks) continue;
                const double bytes = double(p.part_bytes());
                if (p.tail() > 0 && bytes > double(part_bytes)) continue;
                if (S > 1 && sps < 4) continue;
                double us = run_us(p.head, stages) + run_us(double(p.tail()) * S, sps);
                if (p.tail() > 0) us += costs.cut + costs.cut_mb * bytes * 1e-6;
                if (us < best_us) {
                    best_us = us;
                    best = p;
                }
            }
        }
    }
    return best;
}

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
size_t block_fwd_part_bytes(int M, int rows, int K, bool gated);  // for any group size
bool block_fwd_fits(int M, int out, bool gated);                  // whether a launch covers the tiles
wq_status block_fwd(const BlockFwd& p, float* part, size_t part_bytes, hipStream_t s);

// Small M (decode batches): as far as two 16-row fragments of x fit the
// registers.  Up to there the decode kernel is the faster one at every width:
// at 32 rows, 4 bits, groups of 128, 11.9 us against the tile kernel's 16.8 for
// 4096 x 4096, 20.5 against 21.1 for 4096 x 11008 (the closest; 25.2 and 26.7
// at 8 bits), 22.8 against 33.3 for gated 11008 x 4096.  K of more than 64
// ranges of what a block's registers hold of x is the tile kernel's, and so are
// its bytes.
constexpr int kBlockSmallM = 32;
size_t block_small_part_bytes(int M, int rows, int K, int bits, bool gated);
// WQ_ERR_UNSUPPORTED when K has to be split and `part` has no room for it.
wq_status block_small(const BlockFwd& p, float* part, size_t part_bytes, hipStream_t s);

// e applied to the sum over `splits` partial products [splits][M][rows].
wq_status block_finish(const wq::Epilogue& e, bool gated, const float* part, int splits, int M, hipStream_t s);

}  // namespace wqh
