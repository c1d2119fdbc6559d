// The block's forward products for small batches (M <= 32).
//
// y = epilogue(x . W^T) is bound by the weight stream here (2 M flops per
// half byte of 4-bit codes), so the kernel reads every packed word once,
// decodes it in registers and hands the product to the matrix cores, whose
// 16 (or 2 x 16) rows cover all of x.
//
// One v_mfma_f32_16x16x32_f16 takes 16 rows of x and 16 weight rows over 32
// channels: lane l supplies row l % 16 of both, 8 consecutive channels of its
// quarter l / 16.  A lane works on whole chunks (32 codes, four 8-code
// blocks): chunk 4 h + l / 16 of a 128-channel half step h feeds four
// instructions, x is read with the same channel mapping.
//
//  - A block keeps its part of K for all its output tiles (16 weight rows;
//    gated: 16 gate rows and the 16 up rows of the same columns, which meet
//    in the epilogue), cut into one slice per wavefront.  A wavefront's slice
//    of x stays in its registers from start to end, in the order in which the
//    decoder exposes codes (i, i + 4), so x is read once per block and the
//    decoder takes 5 instructions per word.
//  - The packed words of a wavefront's next step (256 channels, 128 at 8
//    bits) are copied from memory into an LDS slot of its own while it
//    decodes the current one from registers, across tile borders, with one
//    wait per step and no barrier, whole lines at a time (eight lanes to 128
//    bytes of a row).  Two and four steps ahead measured equal or slower
//    (2 x 11008 x 4096 at one row: 14.3 us one ahead, 14.5 two).
//  - WIDE: the scales and zero-points of a tile's 16 rows lie together in
//    memory; the block copies them 16 bytes a lane, a tile ahead.  (Copied by
//    each wavefront for its own steps, 2 and 1 bytes a lane, they cost 2 x
//    14336 x 8192 at 8 rows 37 us against 31 without them.)  Layers whose
//    scales are not 16-byte aligned at the tiles or too many for LDS still
//    take that way.
//  - At the end of a tile the wavefronts' partial products meet in LDS in a
//    fixed order (two buffers: one barrier per tile).
// Measured (a pass in a captured graph, three sets of inputs in turn): one row
// of 2 x 11008 x 4096 13.8 us (3.3 TB/s of packed words), 8 rows of 2 x 14336
// x 8192 34.8 us (3.4 TB/s; 31 when the same weights come again, from the
// Infinity Cache), 16 rows of 4096 x 11008 16.1 us with its sums, one row of
// 4096 x 4096 6.0 us.  Start and end take some 5 us of each; in between the
// decoder's vector instructions (13 for 8 codes at 4 bits) bound it, then the
// copies' latency, and tiles that do not fill whole rounds (896 of 2 x 14336
// columns are 3.5 rounds of 256 blocks and take 4).  Placing the scales so that
// their reads do not share banks changed no time.
// (With the stream through double-buffered registers instead, one token
// through 2 x 11008 x 4096 took 27 us, 16 tokens through 4096 x 11008 25 us.)
#include <algorithm>
#include <type_traits>

#include "wq_block_common.h"

namespace {

using namespace wq;

struct SmallArgs {
    const uint16_t* x;
    const uint32_t* packed;
    const uint16_t* scales;
    const uint8_t* zeros;
    float* part;  // fp32 sums of a K split, or null
    int M, rows, K;
    GroupDiv gd;
    int tiles, sps;  // sps: steps of a block's part of K
    Epilogue e;
};

// Pairs (i, i + 4) of an 8-code block as exact fp16 integers B + q: B = 1024
// for the pairs 0 and 2, 64 at 4 bits (codes left at bits 4..7) or 1024 for 1
// and 3.
template <int BITS>
__device__ __forceinline__ void decode_block_pairs(const uint32_t* w, int b, uint32_t (&h)[4]) {
    if constexpr (BITS == 4) {
        const uint32_t v = w[b], v8 = v >> 8;
        h[0] = and_or(v, 0x000F000Fu, kMagic2);
        h[1] = and_or(v, 0x00F000F0u, 0x54005400u);
        h[2] = and_or(v8, 0x000F000Fu, kMagic2);
        h[3] = and_or(v8, 0x00F000F0u, 0x54005400u);
    } else {
        uint32_t all[16];
        decode_chunk<BITS>(w, all);  // the unused blocks' code is dropped
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = all[4 * b + i];
    }
}

template <int BITS, bool WIDE, int T>
struct SmallShape {
    static constexpr int HALVES = BITS == 8 ? 1 : 2;                 // 128-channel halves of a step
    static constexpr int WCOPIES = BITS == 2 ? 1 : 2;                // 1 KB copies of a tile's step
    static constexpr int SCOPIES = WIDE ? 0 : 2 * HALVES;            // scales and zero-points
    static constexpr int TILE = WCOPIES * 1024 + SCOPIES * 256;      // bytes of a tile's step in LDS
    static constexpr int SLOT = T * TILE;
};

// MF: 16-row fragments of x; H: 128-channel halves of x in a wavefront's
// registers; W: wavefronts; gated: T = 2 tiles (gate, up), linear T = 1.
template <int BITS, bool WIDE, int MF, int H, int W, bool GATED>
__global__ void __launch_bounds__(64 * W) block_small_kernel(const SmallArgs p) {
    constexpr int T = GATED ? 2 : 1;
    using Sh = SmallShape<BITS, WIDE, T>;
    constexpr int HALVES = Sh::HALVES, S = H / HALVES;  // steps of a wavefront, at most
    static_assert(H % HALVES == 0, "whole steps");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    // [W] slots, [2][W][T * MF][256] floats, WIDE: [2] tiles' scales and zero-points
    float* const red = reinterpret_cast<float*>(lds + W * Sh::SLOT);
    uint8_t* const meta = lds + W * Sh::SLOT + 2 * W * T * MF * 1024;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int li = lane & 15, lg = lane >> 4;
    const int chunks = p.K / 32;
    const int G = chunk_group(chunks - 1, p.gd) + 1;
    constexpr int STEP = 4 * HALVES;  // chunks of a step
    const int steps = (chunks + STEP - 1) / STEP;
    // this block's steps of K (blockIdx.y), dealt to the wavefronts in
    // contiguous slices
    const int s_block = int(blockIdx.y) * p.sps;
    const int s_count = min(p.sps, steps - s_block);
    const int per = (s_count + W - 1) / W;  // <= S
    const int s0 = s_block + wave * per;
    const int mine = max(0, min(per, s_block + s_count - s0));
    const int half = p.rows / 2;
    const int my_tiles = (p.tiles - int(blockIdx.x) + int(gridDim.x) - 1) / int(gridDim.x);
    const int items = my_tiles * mine;
    const uint32_t row_bytes = uint32_t(chunks) * BITS * 4u;

    // ---- the stream.  A copy's lane reads 16 bytes (12 at 3 bits) of row
    // w_row at w_unit, which undoes the slot's permutation:
    //   3, 4 bits: 8 chunks to a row, chunk u of row r at u ^ ((r / 2) % 8);
    //   8 bits: 8 half chunks to a row (4 chunks), the same;
    //   2 bits: 4 chunk pairs to a row, pair u at u ^ ((r / 4) % 4).
    constexpr int UNIT = BITS == 3 ? 12 : 16;
    constexpr int PER_ROW = BITS == 2 ? 4 : 8;
    const uint32_t w_row = uint32_t(lane) / PER_ROW, w_pos = uint32_t(lane) % PER_ROW;
    const uint32_t w_unit = BITS == 2 ? w_pos ^ ((w_row >> 2) & 3u) : w_pos ^ ((w_row >> 1) & 7u);
    uint8_t* const slot = lds + wave * Sh::SLOT;
    int it = blockIdx.x, is = 0, left = items;  // issue cursor
    u4 wsrc[T], ssrc[T], zsrc[T];                           // of the cursor's tile
    auto first_row = [&](int t, int j) { return 16 * t + (GATED && j ? half : 0); };
    auto rows_from = [&](int n0) { return uint64_t(max(0, p.rows - n0)); };
    auto aim = [&]() {
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const int n0 = first_row(it, j);
            const uint64_t left_rows = rows_from(n0);
            wsrc[j] = copy_source(reinterpret_cast<const char*>(p.packed) + size_t(n0) * row_bytes,
                                  left_rows * row_bytes);
            if constexpr (!WIDE) {
                ssrc[j] = copy_source(p.scales + size_t(n0) * G, left_rows * G * 2);
                zsrc[j] = copy_source(p.zeros ? p.zeros + size_t(n0) * G : nullptr, p.zeros ? left_rows * G : 0);
            }
        }
    };
    // WIDE: tile t's scales (16 G of 2 bytes) and zero-points (16 G bytes), in
    // pieces of 1 KB dealt to the wavefronts, into the buffer of its parity
    const int s_pieces = (32 * G + 1023) / 1024, z_pieces = (16 * G + 1023) / 1024;
    const uint32_t meta_tile = uint32_t(s_pieces + z_pieces) * 1024u;  // of one j
    auto copy_meta = [&](int t, int parity) {
        const uint32_t dst = lds_address(meta) + uint32_t(parity) * T * meta_tile;
        for (int k = wave; k < T * (s_pieces + z_pieces); k += W) {
            const int j = T == 2 && k >= s_pieces + z_pieces ? 1 : 0, q = k - j * (s_pieces + z_pieces);
            const int n0 = first_row(t, j);
            const uint64_t n = rows_from(n0) * G;
            if (q < s_pieces)
                copy_to_lds<16>(copy_source(p.scales + size_t(n0) * G, n * 2), uint32_t(q) * 1024u + lane * 16u,
                                dst + uint32_t(k) * 1024u);
            else if (p.zeros)
                copy_to_lds<16>(copy_source(p.zeros + size_t(n0) * G, n), uint32_t(q - s_pieces) * 1024u + lane * 16u,
                                dst + uint32_t(k) * 1024u);
        }
    };
    // a row's units past K are the next row's codes: their scale is zero, so
    // that they stay finite, and they meet zeros of x
    const uint32_t w_off0 = w_row * row_bytes + w_unit * UNIT;
    const uint32_t w_off1 = (w_row + 8u) * row_bytes + (w_unit ^ 4u) * UNIT;  // (r / 2) % 8 of rows 8 on
    auto issue = [&]() {
        const uint32_t dst = lds_address(slot);
        const uint32_t step = uint32_t(s0 + is);
        uint32_t at[HALVES], at2[HALVES];
        if constexpr (!WIDE) {
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                const int ch = int(step) * STEP + 4 * h + lg;
                at[h] = uint32_t(li) * uint32_t(G) + uint32_t(chunk_group(min(ch, chunks - 1), p.gd));
                at2[h] = ch < chunks ? at[h] * 2u : kNowhere;
            }
        }
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const uint32_t so = step * (PER_ROW * UNIT), d = dst + j * Sh::TILE;
            copy_to_lds<UNIT>(wsrc[j], w_off0 + so, d);
            if constexpr (Sh::WCOPIES == 2) copy_to_lds<UNIT>(wsrc[j], w_off1 + so, d + 1024u);
            if constexpr (!WIDE) {
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    const uint32_t sd = d + Sh::WCOPIES * 1024u + h * 512u;
                    copy_to_lds<2>(ssrc[j], at2[h], sd);
                    copy_to_lds<1>(zsrc[j], at[h], sd + 256u);
                }
            }
        }
        --left;
        if (++is == mine) {
            is = 0;
            it += gridDim.x;
            aim();
        }
    };

    // ---- x: rows li + 16 f (rows past M repeat the last one: their outputs
    // are not stored), zeros past K
    u4 xr[H][4][MF];
    {
        const int c_end = min(chunks, (s0 + mine) * STEP);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int ch = s0 * STEP + 4 * h + lg;
            const bool in = ch < c_end;
#pragma unroll
            for (int f = 0; f < MF; ++f) {
                const u4* xp = reinterpret_cast<const u4*>(p.x + size_t(min(li + 16 * f, p.M - 1)) * p.K +
                                                           32 * size_t(min(ch, chunks - 1)));
#pragma unroll
                for (int q = 0; q < 4; ++q) xr[h][q][f] = in ? xp[q] : u4{0u, 0u, 0u, 0u};
            }
        }
    }
    if constexpr (WIDE) copy_meta(blockIdx.x, 0);
    if (left > 0) {
        aim();
        issue();
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int f = 0; f < MF; ++f) xr[h][q][f] = stage_block(xr[h][q][f]);

    f4 acc[T][MF];
    // One item: its words into registers, its slot to the next item, then
    // decode and multiply by x's halves hs, hs + 1.
    auto work = [&](auto hs_c, int parity) {
        constexpr int hs = decltype(hs_c)::value;
        uint32_t w[T][HALVES][BITS], ss[T][HALVES], zz[T][HALVES];
        copies_landed<0>();
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const uint8_t* t = slot + j * Sh::TILE;
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                const uint32_t ch = 4u * h + lg;
                if constexpr (BITS == 8) {
                    const uint32_t sw = uint32_t(li >> 1) & 7u;
                    const u4 a = *reinterpret_cast<const u4*>(t + li * 128 + ((2u * ch) ^ sw) * 16u);
                    const u4 b = *reinterpret_cast<const u4*>(t + li * 128 + ((2u * ch + 1u) ^ sw) * 16u);
                    w[j][h][0] = a.x; w[j][h][1] = a.y; w[j][h][2] = a.z; w[j][h][3] = a.w;
                    w[j][h][4] = b.x; w[j][h][5] = b.y; w[j][h][6] = b.z; w[j][h][7] = b.w;
                } else if constexpr (BITS == 2) {
                    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
                    const u2 a = *reinterpret_cast<const u2*>(t + li * 64 + ((ch >> 1) ^ (uint32_t(li >> 2) & 3u)) * 16u +
                                                              (ch & 1u) * 8u);
                    w[j][h][0] = a.x; w[j][h][1] = a.y;
                } else {
                    const u4 a = *reinterpret_cast<const u4*>(t + li * 128 + (ch ^ (uint32_t(li >> 1) & 7u)) * 16u);
                    w[j][h][0] = a.x; w[j][h][1] = a.y; w[j][h][2] = a.z;
                    if constexpr (BITS == 4) w[j][h][3] = a.w;
                }
                if constexpr (WIDE) {
                    const uint8_t* mt = meta + (parity * T + j) * meta_tile;
                    const int kc = (s0 + hs / HALVES) * STEP + int(ch);
                    const int g = chunk_group(min(kc, chunks - 1), p.gd);
                    const uint32_t sc = reinterpret_cast<const uint16_t*>(mt)[li * G + g];
                    ss[j][h] = kc < chunks ? sc : 0u;
                    zz[j][h] = mt[s_pieces * 1024 + li * G + g];
                } else {
                    const uint32_t* sp = reinterpret_cast<const uint32_t*>(t + Sh::WCOPIES * 1024 + h * 512);
                    ss[j][h] = sp[lane];
                    zz[j][h] = sp[64 + lane];
                }
            }
        }
        // the reads have left the slot before the copies may enter it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (left > 0) issue();
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            uint32_t ze[T], zo[T], sp[T];
#pragma unroll
            for (int j = 0; j < T; ++j) {
                const uint32_t z = p.zeros ? zz[j][h] : 1u << (BITS - 1);
                ze[j] = zero_pair(z);
                zo[j] = BITS == 4 ? (0x5400u | (z << 4)) * 0x10001u : ze[j];
                sp[j] = scale_pair(uint16_t(ss[j][h]));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
#pragma unroll
                for (int j = 0; j < T; ++j) {
                    uint32_t v[4];
                    decode_block_pairs<BITS>(w[j][h], q, v);
                    v[0] = as_u32(dequant_pair(v[0], ze[j], sp[j]));
                    v[1] = as_u32(dequant_pair(v[1], zo[j], sp[j]));
                    v[2] = as_u32(dequant_pair(v[2], ze[j], sp[j]));
                    v[3] = as_u32(dequant_pair(v[3], zo[j], sp[j]));
                    const h8 b = __builtin_bit_cast(h8, (u4{v[0], v[1], v[2], v[3]}));
#pragma unroll
                    for (int f = 0; f < MF; ++f)
                        acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            __builtin_bit_cast(h8, xr[hs + h][q][f]), b, acc[j][f], 0, 0, 0);
                }
            }
        }
    };

    // the tile's partial products meet: lane l holds rows 4 (l / 16) + r of
    // column l % 16; thread o finishes output (o / 16, o % 16)
    static_assert(16 * 16 * MF <= 64 * W, "one output per thread");
    const int o = threadIdx.x;
    auto tile_end = [&](int t, int parity) {
        float* mine_at = red + (parity * W + wave) * (T * MF * 256);
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
            for (int f = 0; f < MF; ++f) *reinterpret_cast<f4*>(mine_at + (j * MF + f) * 256 + lane * 4) = acc[j][f];
        __syncthreads();
        {
            const int nn = o & 15, m = o >> 4;
            if (m >= p.M) return;
            const float* src = red + parity * W * (T * MF * 256) + (m >> 4) * 256 +
                               (16 * ((m & 15) >> 2) + nn) * 4 + (m & 3);
            float a[1] = {0.f}, u[1] = {0.f};
#pragma unroll
            for (int w = 0; w < W; ++w) {
                a[0] += src[w * (T * MF * 256)];
                if constexpr (GATED) u[0] += src[w * (T * MF * 256) + MF * 256];
            }
            const int col = 16 * t + nn;
            if (col >= p.e.out) return;
            if (p.part) {
                float* dst = p.part + (size_t(blockIdx.y) * p.M + m) * p.rows + col;
                dst[0] = a[0];
                if constexpr (GATED) dst[half] = u[0];
            } else {
                finish<GATED, 1>(p.e, m, col, a, u);
            }
        }
    };

    if constexpr (WIDE) {
        copies_landed<0>();
        __syncthreads();
    }
    for (int k = 0; k < my_tiles; ++k) {
        const int t = int(blockIdx.x) + k * int(gridDim.x), par = k & 1;
        // (the other parity's reads ended before the last barrier)
        if constexpr (WIDE) copy_meta(t + int(gridDim.x), par ^ 1);
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
            for (int f = 0; f < MF; ++f) acc[j][f] = f4{0.f, 0.f, 0.f, 0.f};
        // (the steps are unrolled: x's registers are named at compile time)
        if (0 < mine) work(std::integral_constant<int, 0>{}, par);
        if constexpr (S > 1) if (1 < mine) work(std::integral_constant<int, HALVES>{}, par);
        if constexpr (S > 2) if (2 < mine) work(std::integral_constant<int, 2 * HALVES>{}, par);
        if constexpr (S > 3) if (3 < mine) work(std::integral_constant<int, 3 * HALVES>{}, par);
        static_assert(S <= 4, "steps of a wavefront");
        // (the next tile's scales have landed: an item's wait came after their
        // copies)
        if (WIDE && mine == 0) copies_landed<0>();
        tile_end(t, par);
    }
    copies_landed<0>();  // none may still be writing when the block ends
}

constexpr int kSmallLds = 160 * 1024;

// Launch shape: the smallest slice of x that K's steps fit in, K split across
// blocks where they fit in none, or where the tiles alone leave compute units
// without work.
struct SmallPlan {
    int H = 2, W = 8, tiles = 0, blocks = 0, splits = 1, sps = 0;
    int meta_tile = 0;  // LDS bytes of a tile's scales and zero-points
    bool ok = false, wide = false;
};

SmallPlan small_plan(int M, int rows, int K, int bits, bool gated, size_t part_bytes) {
    SmallPlan p;
    const int cus = wqh::gemm_slots(1);
    const int halves = bits == 8 ? 1 : 2;
    const int steps = (K / 32 + 4 * halves - 1) / (4 * halves);
    p.tiles = gated ? (rows / 2 + 15) / 16 : (rows + 15) / 16;
    // halves of x per block: 16 wavefronts of up to 4 (one fragment of rows),
    // or 8 of up to 4 (two)
    const int most = (M > 16 ? 8 : 16) * 4;
    const size_t copy = size_t(M) * rows * 4;
    const int afford = copy ? int(std::min<size_t>(part_bytes / copy, 64)) : 1;
    int S = (steps * halves + most - 1) / most;
    // A range takes at least 16 steps, which suits one row: 1024 x 8192 7.4 us
    // in the two ranges of this rule, 7.6 whole; 1024 x 4096 5.1 whole, 6.0 in
    // two; 2048 x 8192 8.2 in two, 7.9 whole.  More rows would take more ranges
    // (1024 x 8192 at 32 rows: 14.0 us in two, 10.5 in four).
    while (S < afford && p.tiles * (S + 1) <= cus && steps >= 16 * (S + 1)) ++S;
    if (S > 1 && S > afford) return p;
    p.sps = (steps + S - 1) / S;
    p.splits = (steps + p.sps - 1) / p.sps;
    const int need = p.sps * halves;  // halves of x per block
    p.W = M > 16 || need <= 16 ? 8 : 16;
    p.H = need <= 2 * p.W ? 2 : 4;
    p.blocks = std::min(p.tiles, std::max(1, cus / p.splits));
    p.ok = true;
    return p;
}

template <int BITS, bool WIDE, int MF, int H, int W, bool GATED>
wq_status launch_small(const SmallPlan& pl, const SmallArgs& a, hipStream_t s) {
    constexpr int T = GATED ? 2 : 1;
    constexpr int fixed = W * SmallShape<BITS, WIDE, T>::SLOT + 2 * W * T * MF * 1024;
    static_assert(fixed <= kSmallLds, "LDS");
    const int lds = fixed + (WIDE ? 2 * T * pl.meta_tile : 0);
    if (lds > kSmallLds) return launch_small<BITS, false, MF, H, W, GATED>(pl, a, s);
    auto kern = block_small_kernel<BITS, WIDE, MF, H, W, GATED>;
    // (the limit is the process's, not the call's: one value for every call, or
    // a thread with a smaller layer could lower it under another's launch)
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kSmallLds);
    if (e != hipSuccess) return wqh::hip_status(e);
    hipLaunchKernelGGL(kern, dim3(pl.blocks, pl.splits), dim3(64 * W), lds, s, a);
    return wqh::launch_status();
}

template <int BITS, bool WIDE, bool GATED>
wq_status launch_small_shape(const SmallPlan& pl, const SmallArgs& a, hipStream_t s) {
    if (a.M > 16)
        return pl.H == 2 ? launch_small<BITS, WIDE, 2, 2, 8, GATED>(pl, a, s) : launch_small<BITS, WIDE, 2, 4, 8, GATED>(pl, a, s);
    if (pl.W == 8) return launch_small<BITS, WIDE, 1, 2, 8, GATED>(pl, a, s);
    return pl.H == 2 ? launch_small<BITS, WIDE, 1, 2, 16, GATED>(pl, a, s)
                     : launch_small<BITS, WIDE, 1, 4, 16, GATED>(pl, a, s);
}

template <int BITS>
wq_status launch_small_bits(const wqh::BlockFwd& f, const SmallPlan& pl, const SmallArgs& a, hipStream_t s) {
    if (f.gated)
        return pl.wide ? launch_small_shape<BITS, true, true>(pl, a, s) : launch_small_shape<BITS, false, true>(pl, a, s);
    return pl.wide ? launch_small_shape<BITS, true, false>(pl, a, s) : launch_small_shape<BITS, false, false>(pl, a, s);
}

}  // namespace

namespace wqh {

size_t block_small_part_bytes(int M, int rows, int K, int bits, bool gated) {
    const SmallPlan p = small_plan(M, rows, K, bits, gated, ~size_t(0));
    if (!p.ok) return block_fwd_part_bytes(M, rows, K, gated);  // the tile kernel takes the call
    return p.splits > 1 ? size_t(p.splits) * M * rows * 4 : 0;
}

wq_status block_small(const BlockFwd& f, float* part, size_t part_bytes, hipStream_t s) {
    SmallPlan pl = small_plan(f.M, f.rows, f.K, f.bits, f.gated, part ? part_bytes : 0);
    if (!pl.ok) return WQ_ERR_UNSUPPORTED;
    // every tile's scales and zero-points start and end on 16 bytes
    const size_t G = size_t(f.K / f.gs), half = f.gated ? size_t(f.rows / 2) : 0;
    pl.wide = aligned16(f.scales) && aligned16(f.zeros) && size_t(f.rows) * G % 16 == 0 && half * G % 16 == 0;
    pl.meta_tile = int((32 * G + 1023) / 1024 + (16 * G + 1023) / 1024) * 1024;
    const SmallArgs a{f.x, f.packed, f.scales, f.zeros, pl.splits > 1 ? part : nullptr, f.M, f.rows, f.K,
                      group_magic(f.gs), pl.tiles, pl.sps, f.e};
    wq_status st;
    switch (f.bits) {
        case 2: st = launch_small_bits<2>(f, pl, a, s); break;
        case 3: st = launch_small_bits<3>(f, pl, a, s); break;
        case 4: st = launch_small_bits<4>(f, pl, a, s); break;
        default: st = launch_small_bits<8>(f, pl, a, s); break;
    }
    if (st != WQ_OK || pl.splits == 1) return st;
    return block_finish(f.e, f.gated, part, pl.splits, f.M, s);
}

}  // namespace wqh
