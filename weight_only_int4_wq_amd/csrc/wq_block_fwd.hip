// The block's forward products for more rows than a decode batch:
// epilogue(x . W^T) on 32x32x16 fp16 matrix-core instructions.
//
// A 256-thread block owns BM activation rows x 256 weight rows of products;
// its four wavefronts sit side by side along the weight rows, BM x 64 each, so
// that every weight is decoded by one wavefront only, and the vector work of
// decoding is spread over BM / 32 matrix instructions per fragment.  K
// advances in stages of 64.
//
//  - Weights: lane l supplies 8 consecutive channels (half l / 32 of the
//    stage's 64) of one weight row, which is one packed 8-code block.  The
//    packed codes pass through LDS in windows of GS stages (64 bytes of a
//    row, 48 at 3 bits), copied with four lanes to a row, scales and
//    zero-points in windows of their own: lanes that load their own chunk,
//    scale and zero-point per stage straight from memory fetch a whole line
//    for each of them every time.  A lane reads its 32-code chunk, scale and
//    zero-point from LDS once per stage and dequantizes in registers straight
//    into the B operand.
//  - The lane's two weight rows are neighbours (2c, 2c + 1) in the linear
//    layer, and gate row o with up row o + I in the gated block: both
//    factors of an output then sit in the same lane's accumulators.
//  - Activations: three LDS buffers of BM x 64; stage s + 2 is on its way
//    while stage s is multiplied.
//  - All of it is copied from memory straight into LDS, and each stage ends
//    with one wait that leaves the newest stage's copies in flight.  (4096 x
//    8192 x 8192 at 4 bits: 535 us; with loads through registers 553, of
//    which 428 are left without any loads and 374 with nothing but the matrix
//    instructions.)
//  - Epilogue: accumulators cross LDS in passes of 64 rows, so that bias,
//    activation, product, residual and every store work on 8 neighbouring
//    columns (16-byte accesses).
//  - Tiles are dealt to the XCDs in contiguous ranges (tile_work).  What a last,
//    partly filled round of tiles leaves idle is used by cutting those tiles
//    along K: 2048 x 11008 x 4096, 128 tiles, in two ranges 178 us, whole
//    204 us.
//  Measured: 2048 x 4096 x 2 x 11008 at 4 bits, gated, 364-369 us a pass (1000
//  TFLOP/s; the card's matrix units are held back by power there: the loop's
//  matrix instructions alone reach 1470).
#include <algorithm>
#include <type_traits>

#include "wq_block_common.h"

namespace {

using namespace wq;

// Vector instructions issued after each matrix instruction.
#ifndef WQ_BLOCK_FWD_VALU
#define WQ_BLOCK_FWD_VALU 4
#endif

struct FwdArgs {
    const uint16_t* x;
    const uint32_t* packed;
    const uint16_t* scales;
    const uint8_t* zeros;
    float* part;  // [ranges][tail tiles][BM][256] partial products
    int M, rows, K;
    GroupDiv gd;
    int m_tiles, n_tiles, tiles, head, sps;
    int gated;
    Epilogue e;
};

// Shape of the tile kernel's shared memory.
template <int BITS, bool FAST, int BM>
struct FwdShape {
    static constexpr int BK = 64;
    static constexpr int GS = BITS == 8 ? 1 : BITS == 2 ? 4 : 2;  // stages of a weight window
    static constexpr int UNIT = BITS == 3 ? 12 : 16;              // bytes a lane copies (16 apart in LDS)
    static constexpr int SG = FAST ? 4 : 2;                       // stages of a window of scales
    static constexpr int NS = FAST ? 2 : 4;                       // scales of a row in it
    static constexpr int A_BYTES = BM * BK * 2;
    static constexpr int W_BYTES = 256 * 4 * 16;
    static constexpr int S_BYTES = NS * 2 * 256 * 4;
    static constexpr int PASS = 64;                               // rows of an epilogue pass
    static constexpr int MAIN = 3 * A_BYTES + 2 * (W_BYTES + S_BYTES);
    static constexpr int LDS = MAIN > PASS * 256 * 4 ? MAIN : PASS * 256 * 4;
};

// Outputs oc .. oc + 7 of a tile row.  The tile's column 32 w + c holds the
// first and 128 + 32 w + c the second weight row of lane c of wavefront w: the
// gate's and the up projection's of output 32 w + c, or columns 64 w + 2 c and
// 64 w + 2 c + 1.
// get(at, v): four neighbouring columns of the tile row, per entry of `at`.
template <class Get>
__device__ __forceinline__ void finish_piece(const Epilogue& e, bool gated, bool wide, int row, int o0, int oc,
                                             const Get& get) {
    const int col = o0 + oc;
    if (col >= e.out) return;
    float a[8], u[8];
    if (gated) {
        const int at[4] = {oc, oc + 4, 128 + oc, 132 + oc};
        f4 v[4];
        get(at, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = v[i / 4][i % 4];
            u[i] = v[2 + i / 4][i % 4];
        }
        if (wide) {
            finish<true, 8>(e, row, col, a, u);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float a1[1] = {a[i]}, u1[1] = {u[i]};
                if (col + i < e.out) finish<true, 1>(e, row, col + i, a1, u1);
            }
        }
    } else {
        const int at[2] = {oc / 2, 128 + oc / 2};
        f4 v[2];
        get(at, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = v[i & 1][i >> 1];
            u[i] = 0.f;
        }
        if (wide) {
            finish<false, 8>(e, row, col, a, u);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float a1[1] = {a[i]}, u1[1] = {0.f};
                if (col + i < e.out) finish<false, 1>(e, row, col + i, a1, u1);
            }
        }
    }
}

// FAST: the group size is a multiple of 128 (or all of K, itself a multiple),
// so two stages share a scale and zero-point.
template <int BITS, bool FAST, int BM>
__global__ void __launch_bounds__(256, 1) block_fwd_kernel(const FwdArgs p) {
    using Sh = FwdShape<BITS, FAST, BM>;
    constexpr int BN = 256, BK = Sh::BK, TM = BM / 32, TN = 2;
    constexpr int GS = Sh::GS, SG = Sh::SG, NS = Sh::NS, UNIT = Sh::UNIT;
    constexpr int ROW = BK * 2;  // bytes of an activation row in LDS
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Sh::LDS];
    uint8_t* const lds_a = lds;                       // [3][BM][64]
    uint8_t* const lds_w = lds_a + 3 * Sh::A_BYTES;   // [2][256 rows][4 units]
    uint8_t* const lds_s = lds_w + 2 * Sh::W_BYTES;   // [2][NS][scale, zero-point][256 rows]

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 31, hh = lane >> 5;
    const bool gated = p.gated != 0;
    const int oc_tile = gated ? BN / 2 : BN;  // output columns of the tile
    const TileWork tw = tile_work(blockIdx.x, p.tiles, p.head, p.m_tiles, p.n_tiles);
    const int m0 = tw.m_t * BM, o0 = tw.n_t * oc_tile;
    const int chunks = p.K / 32;
    const int G = chunk_group(chunks - 1, p.gd) + 1;
    const int stages = (p.K + BK - 1) / BK;
    const int st_begin = tw.split * p.sps;  // a multiple of 4
    const int st_end = tw.part < 0 ? stages : min(st_begin + p.sps, stages);

    const TileCopy<BM> xcopy(p.x + size_t(m0) * p.K, p.M - m0, p.K, wave, lane);

    // ---- weights.  LDS row r = 128 j + 32 w + c is what lane c of wavefront w
    // multiplies as its j-th row: gate (j = 0) or up row o0 + 32 w + c, or row
    // o0 + 64 w + 2 c + j.  Wavefront k copies LDS rows 64 k .. 64 k + 63, all
    // of one j, from the matrix row `first` on (rows past the matrix become
    // zeros or other rows; their outputs are not stored).
    const int kj = wave >> 1, kh = wave & 1;
    const int first = o0 + (gated ? kj * p.e.out : kj);
    const uint32_t row_bytes = uint32_t(chunks) * BITS * 4u;
    const int rows_left = p.rows - first;  // may be <= 0
    auto left = [&](uint64_t per_row) { return rows_left > 0 ? uint64_t(rows_left) * per_row : 0; };
    const u4 wsrc = copy_source(reinterpret_cast<const char*>(p.packed) + size_t(first) * row_bytes, left(row_bytes));
    // Part cp = 0 .. 3 of a window: LDS rows 64 k + 16 cp + l / 4, lane l the
    // row's position l % 4, which holds unit (l % 4) ^ ((row / 4) % 4): 16
    // consecutive rows read at one unit fall on all banks.
    const uint32_t wstep = (gated ? 16u : 32u) * row_bytes;
    const uint32_t wunit = uint32_t(lane & 3) ^ uint32_t(lane >> 4);
    const uint32_t woff = (gated ? 64u * kh + uint32_t(lane >> 2) : 128u * kh + 2u * uint32_t(lane >> 2)) * row_bytes +
                          wunit * UNIT;
    // Parts GS-th by GS-th in one sequence over the stages: the Q-th belongs
    // to window Q / GS.
    constexpr int WP = 4 / GS;  // parts a stage copies
    auto copy_w = [&](int Q) {
        const uint32_t off = woff + uint32_t(Q / GS) * (4u * UNIT);
        const uint32_t cp0 = uint32_t(Q & (GS - 1)) * WP;
        const uint32_t dst = lds_address(lds_w + ((Q / GS) & 1) * Sh::W_BYTES) + (64u * wave + 16u * cp0) * 64u;
#pragma unroll
        for (int e = 0; e < WP; ++e) copy_to_lds<UNIT>(wsrc, off + (cp0 + e) * wstep, dst + e * 1024u);
    };
    // Scales and zero-points: thread t copies LDS row t's; scales past K are
    // zero (the codes there are the next row's, and meet zeros of x).
    const u4 ssrc = copy_source(p.scales + size_t(first) * G, left(uint64_t(G) * 2));
    const u4 zsrc = copy_source(p.zeros ? p.zeros + size_t(first) * G : nullptr, p.zeros ? left(G) : 0);
    const uint32_t soff = (gated ? 64u * kh + uint32_t(lane) : 128u * kh + 64u * uint32_t(lane >> 5) + 2u * c) * uint32_t(G);
    auto copy_s = [&](int g) {
        const uint32_t dst = lds_address(lds_s + (g & 1) * Sh::S_BYTES) + 256u * wave;
#pragma unroll
        for (int q = 0; q < NS; ++q) {
            const int ch = (g * SG * 2) + q * (SG * 2 / NS);
            const uint32_t at = soff + uint32_t(chunk_group(min(ch, chunks - 1), p.gd));
            copy_to_lds<2>(ssrc, ch < chunks ? at * 2u : kNowhere, dst + q * 2048u);
            copy_to_lds<1>(zsrc, at, dst + q * 2048u + 1024u);
        }
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    // The k-steps of a stage are software-pipelined: while k-step t's matrix
    // instructions run, the A fragments of t + 1 are read and its B fragments
    // decoded.  The stage's barrier sits before its last k-step, whose
    // instructions then cover the first reads of the next stage's buffers.
    const uint32_t a_lane = uint32_t(c) * ROW;
    const uint32_t w_lane = uint32_t(wave) * 32u + uint32_t(c);  // LDS row of j = 0
    h8 af[2][TM], bf[2][TN];
    uint32_t wc[TN][BITS], zz[TN], ss[TN];  // the stage's chunk of each row
    auto read_w = [&](int st) {
        const uint32_t i = uint32_t(st) & (GS - 1);
        const uint8_t* win = lds_w + ((st / GS) & 1) * Sh::W_BYTES;
        const uint32_t q = FAST ? uint32_t(st >> 1) & 1u : 2u * (uint32_t(st) & 1u) + hh;
        const uint32_t* s = reinterpret_cast<const uint32_t*>(lds_s + ((st / SG) & 1) * Sh::S_BYTES) + q * 512u;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const uint32_t r = w_lane + 128u * j, sw = (r >> 2) & 3u;
            const uint8_t* row = win + r * 64u;
            if constexpr (BITS == 4) {
                const u4 v = *reinterpret_cast<const u4*>(row + ((2u * i + hh) ^ sw) * 16u);
                wc[j][0] = v.x; wc[j][1] = v.y; wc[j][2] = v.z; wc[j][3] = v.w;
            } else if constexpr (BITS == 8) {
                const u4 a = *reinterpret_cast<const u4*>(row + ((2u * hh) ^ sw) * 16u);
                const u4 b = *reinterpret_cast<const u4*>(row + ((2u * hh + 1u) ^ sw) * 16u);
                wc[j][0] = a.x; wc[j][1] = a.y; wc[j][2] = a.z; wc[j][3] = a.w;
                wc[j][4] = b.x; wc[j][5] = b.y; wc[j][6] = b.z; wc[j][7] = b.w;
            } else if constexpr (BITS == 2) {
                typedef uint32_t u2 __attribute__((ext_vector_type(2)));
                const u2 v = *reinterpret_cast<const u2*>(row + (i ^ sw) * 16u + hh * 8u);
                wc[j][0] = v.x; wc[j][1] = v.y;
            } else {
                const u4 v = *reinterpret_cast<const u4*>(row + ((2u * i + hh) ^ sw) * 16u);
                wc[j][0] = v.x; wc[j][1] = v.y; wc[j][2] = v.z;
            }
            ss[j] = s[r];
            zz[j] = s[256u + r];
        }
    };
    auto group_pairs = [&]() {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            ss[j] = __builtin_amdgcn_perm(ss[j], ss[j], 0x01000100u);
            zz[j] = zero_pair_nat<BITS>(p.zeros ? zz[j] : 1u << (BITS - 1));
        }
    };
    auto read_a = [&](const uint8_t* buf, int t, h8 (&f)[TM]) {
        const uint8_t* ap = buf + a_lane + ((uint32_t(4 * hh + t) ^ uint32_t((c >> 1) & 7)) * 16u);
#pragma unroll
        for (int i = 0; i < TM; ++i) f[i] = *reinterpret_cast<const h8*>(ap + i * 32 * ROW);
    };
    auto make_b = [&](int t, h8 (&f)[TN]) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            uint32_t hq[4], v[4];
            decode_nat<BITS>(wc[j], t, hq);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = as_u32(dequant_pair(hq[q], zz[j], ss[j]));
            f[j] = __builtin_bit_cast(h8, (u4{v[0], v[1], v[2], v[3]}));
        }
    };
    auto multiply = [&](const h8 (&a)[TM], const h8 (&b)[TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[i], b[j], acc[i][j], 0, 0, 0);
    };
    constexpr int NM = TM * TN, NV = WQ_BLOCK_FWD_VALU;
    constexpr int C = TileCopy<BM>::COPIES;
    auto abuf = [&](int k) { return lds_a + k * Sh::A_BYTES; };

    // ---- the first windows, two stages of x.  Scales' window g + 1 is copied
    // in window g's first stage, the weights' parts one by one.
    copy_s(st_begin / SG);
#pragma unroll
    for (int q = 0; q <= GS; ++q) copy_w(st_begin + q);
    xcopy.copy(xcopy.stage(st_begin, abuf(0)), 0, C);
    xcopy.copy(xcopy.stage(st_begin + 1, abuf(1)), 0, C);
    copies_landed<C>();
    __syncthreads();
    read_w(st_begin);
    read_a(abuf(0), 0, af[0]);
    group_pairs();
    make_b(0, bf[0]);
    int b0 = 0, b1 = 1, b2 = 2;  // buffers of stages st, st + 1, st + 2
    for (int st = st_begin; st < st_end; ++st) {
        // stage st + 2's copies (past K: zeros) into the buffer that every
        // wavefront has left by the last barrier
        const auto next = xcopy.stage(st + 2, abuf(b2));
        const uint8_t* buf = abuf(b0);
        read_a(buf, 1, af[1]);
        make_b(1, bf[1]);
        xcopy.copy(next, 0, (C + 2) / 3);
        multiply(af[0], bf[0]);
        sched_step<NM, TM, 0, 0, NV>();
        read_a(buf, 2, af[0]);
        make_b(2, bf[0]);
        xcopy.copy(next, (C + 2) / 3, (2 * C + 2) / 3);
        multiply(af[1], bf[1]);
        sched_step<NM, TM, 0, 0, NV>();
        read_a(buf, 3, af[1]);
        make_b(3, bf[1]);
        xcopy.copy(next, (2 * C + 2) / 3, C);
        multiply(af[0], bf[0]);
        sched_step<NM, TM, 0, 0, NV>();
        copies_landed<C>();  // all but stage st + 2's
        __syncthreads();
        read_w(st + 1);
        read_a(abuf(b1), 0, af[0]);
        copy_w(st + 1 + GS);  // into a part whose window's last reads lie before this barrier
        group_pairs();
        make_b(0, bf[0]);
        multiply(af[1], bf[1]);
        sched_step<NM, TM + 2 * TN, 0, 0, NV>();
        if ((st & (SG - 1)) == 0) copy_s(st / SG + 1);
        const int t = b0;
        b0 = b1;
        b1 = b2;
        b2 = t;
    }
    copies_landed<0>();  // none may still be writing when LDS is reused or the block ends
    __syncthreads();

    // ---- acc[i][j][r]: row 32 i + 8 (r / 4) + 4 hh + r % 4, the lane's j-th
    // weight row
    if (tw.part >= 0) {
        // columns as the LDS tile below has them; rows and columns past the
        // matrix are written too (the tile is whole) and never read
        float* pr = p.part + size_t(tw.part) * (BM * BN) + wave * 32 + c;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float* dst = pr + (32 * i + 8 * (r >> 2) + 4 * hh + (r & 3)) * BN;
                dst[0] = acc[i][0][r];
                dst[128] = acc[i][1][r];
            }
        return;
    }
    // LDS tile: the wavefront's first rows' products in columns 32 w + c, the
    // second rows' in 128 + 32 w + c
    float* tile = reinterpret_cast<float*>(lds);  // [PASS][BN]
    const bool wide = p.e.out % 8 == 0;
    const int per_row = oc_tile / 8;
    auto pass = [&](auto ps_c) {  // (named at compile time, as the accumulators are)
        constexpr int ps = decltype(ps_c)::value;
        if (ps) __syncthreads();
#pragma unroll
        for (int ii = 0; ii < Sh::PASS / 32; ++ii)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float* dst = tile + (32 * ii + 8 * (r >> 2) + 4 * hh + (r & 3)) * BN + wave * 32 + c;
                dst[0] = acc[ps * (Sh::PASS / 32) + ii][0][r];
                dst[128] = acc[ps * (Sh::PASS / 32) + ii][1][r];
            }
        __syncthreads();
#pragma unroll 1
        for (int q = tid; q < Sh::PASS * per_row; q += 256) {
            const int rr = q / per_row, oc = (q % per_row) * 8;
            const int row = m0 + ps * Sh::PASS + rr;
            if (row < p.M)
                finish_piece(p.e, gated, wide, row, o0, oc, [&](const auto& at, auto& v) {
#pragma unroll
                    for (unsigned i = 0; i < sizeof(at) / sizeof(at[0]); ++i)
                        v[i] = *reinterpret_cast<const f4*>(&tile[rr * BN + at[i]]);
                });
        }
    };
    pass(std::integral_constant<int, 0>{});
    if constexpr (BM > 64) pass(std::integral_constant<int, 1>{});
    if constexpr (BM > 128) {
        pass(std::integral_constant<int, 2>{});
        pass(std::integral_constant<int, 3>{});
    }
}

// The same for tiles cut in ranges: one piece of a tail tile per thread, the
// ranges' partial products added in order; a launch's blocks count from
// `first`.  Bound by reading them: 67 MB in 16 us, two ranges of 2048 x 4096.
// (With a capped grid that loops over the pieces instead: 18.)
template <int BM>
__global__ void __launch_bounds__(256) block_tail_kernel(const FwdArgs p, int splits, int first) {
    const bool gated = p.gated != 0, wide = p.e.out % 8 == 0;
    const int oc_tile = gated ? 128 : 256, per_row = oc_tile / 8, rows = 256 / per_row;
    const int tail = p.tiles - p.head, per_tile = BM / rows, b = first + int(blockIdx.x), i = b / per_tile;
    int m_t, n_t;
    tile_place(p.head + i, p.m_tiles, p.n_tiles, m_t, n_t);
    const int rr = (b % per_tile) * rows + threadIdx.x / per_row, oc = (threadIdx.x % per_row) * 8;
    const int row = m_t * BM + rr;
    if (row >= p.M) return;
    const float* src = p.part + (size_t(i) * BM + rr) * 256;
    finish_piece(p.e, gated, wide, row, n_t * oc_tile, oc, [&](const auto& at, auto& v) {
        sum_ranges(src, at, size_t(tail) * (BM * 256), splits, v);
    });
}

// Epilogue of a split product: V outputs of one row per thread, the ranges'
// partial sums added in order.
template <bool GATED, int V>
__global__ void __launch_bounds__(256) block_finish_kernel(const Epilogue e, const float* __restrict__ part,
                                                           int splits, int M) {
    const int per_row = e.out / V;
    const int rows = GATED ? 2 * e.out : e.out;
    const size_t total = size_t(M) * per_row, step = size_t(M) * rows;
    for (size_t i = size_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += size_t(gridDim.x) * 256) {
        const int row = int(i / per_row), col = int(i % per_row) * V;
        const float* src = part + size_t(row) * rows + col;
        float a[V], u[V];
#pragma unroll
        for (int k = 0; k < V; ++k) a[k] = u[k] = 0.f;
        for (int s = 0; s < splits; ++s, src += step) {
            float v[V];
            __builtin_memcpy(v, __builtin_assume_aligned(src, 4 * V), 4 * V);
#pragma unroll
            for (int k = 0; k < V; ++k) a[k] += v[k];
            if constexpr (GATED) {
                __builtin_memcpy(v, __builtin_assume_aligned(src + e.out, 4 * V), 4 * V);
#pragma unroll
                for (int k = 0; k < V; ++k) u[k] += v[k];
            }
        }
        finish<GATED, V>(e, row, col, a, u);
    }
}

// [FAST].  (Not FAST, a lane fetches a scale and zero-point from LDS for every
// stage, so that fewer, taller tiles pay earlier.)
constexpr wqh::TileCosts kFwdCosts[2] = {
    {{{64, 1.034, 0.619, 0.0, false}, {128, 1.094, 0.483, 1.255, false}, {256, 1.643, 0.529, 2.812, false}},
     8.568, 0.212},
    {{{64, 0.428, 0.42, 10.497, true}, {128, 0.65, 0.589, 9.933, false}, {256, 1.243, 0.337, 14.647, false}},
     0.418, 0.328}};

wqh::TilePlan fwd_plan(int M, int rows, int K, bool gated, bool fast, size_t part_bytes) {
    const int n_tiles = gated ? (rows / 2 + 127) / 128 : (rows + 255) / 256;
    // ranges of whole windows of weights and scales (four stages)
    return wqh::plan_tiles(M, n_tiles, (K + 63) / 64, kFwdCosts[fast], 4, part_bytes, wqh::gemm_slots(1), false);
}

bool fast_groups(int gs) { return gs % 128 == 0; }

template <int BITS, bool FAST, int BM>
wq_status launch_fwd(const wqh::TilePlan& pl, const FwdArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((block_fwd_kernel<BITS, FAST, BM>), dim3(pl.blocks()), dim3(256), 0, s, a);
    const wq_status st = wqh::launch_status();
    if (st != WQ_OK || pl.tail() == 0) return st;
    return wqh::launch_pieces(pl.tail() * (BM / (a.gated ? 16LL : 8LL)), [&](unsigned blocks, int first) {
        hipLaunchKernelGGL((block_tail_kernel<BM>), dim3(blocks), dim3(256), 0, s, a, pl.splits, first);
    });
}

template <int BITS, bool FAST>
wq_status launch_fwd_bm(const wqh::TilePlan& pl, const FwdArgs& a, hipStream_t s) {
    switch (pl.BM) {
        case 64: return launch_fwd<BITS, FAST, 64>(pl, a, s);
        case 128: return launch_fwd<BITS, FAST, 128>(pl, a, s);
        default: return launch_fwd<BITS, FAST, 256>(pl, a, s);
    }
}

template <int BITS>
wq_status launch_fwd_bits(int gs, const wqh::TilePlan& pl, const FwdArgs& a, hipStream_t s) {
    return fast_groups(gs) ? launch_fwd_bm<BITS, true>(pl, a, s) : launch_fwd_bm<BITS, false>(pl, a, s);
}

}  // namespace

namespace wqh {

bool block_fwd_fits(int M, int out, bool gated) {
    const int oc = gated ? 128 : 256;
    return (M + 255LL) / 256 * ((out + oc - 1LL) / oc) <= kMaxBlocks;
}

size_t block_fwd_part_bytes(int M, int rows, int K, bool gated) {
    return std::max(fwd_plan(M, rows, K, gated, false, ~size_t(0)).part_bytes(),
                    fwd_plan(M, rows, K, gated, true, ~size_t(0)).part_bytes());
}

wq_status block_fwd(const BlockFwd& f, float* part, size_t part_bytes, hipStream_t s) {
    const TilePlan pl = fwd_plan(f.M, f.rows, f.K, f.gated, fast_groups(f.gs), part ? part_bytes : 0);
    if (pl.tiles == 0) return WQ_ERR_ARG;
    const int oc = f.gated ? 128 : 256;
    const int m_tiles = (f.M + pl.BM - 1) / pl.BM, n_tiles = (f.e.out + oc - 1) / oc;
    const FwdArgs a{f.x, f.packed, f.scales, f.zeros, part, f.M, f.rows, f.K, group_magic(f.gs), m_tiles, n_tiles,
                    pl.tiles, pl.head, pl.sps, f.gated, f.e};
    switch (f.bits) {
        case 2: return launch_fwd_bits<2>(f.gs, pl, a, s);
        case 3: return launch_fwd_bits<3>(f.gs, pl, a, s);
        case 4: return launch_fwd_bits<4>(f.gs, pl, a, s);
        default: return launch_fwd_bits<8>(f.gs, pl, a, s);
    }
}

wq_status block_finish(const wq::Epilogue& e, bool gated, const float* part, int splits, int M, hipStream_t s) {
    const bool wide = e.out % 4 == 0;
    const size_t total = size_t(M) * e.out / (wide ? 4 : 1);
    const int blocks = int(std::min<size_t>((total + 255) / 256, size_t(gemm_slots(8))));
    const dim3 g(blocks), b(256);
    if (gated && wide)
        hipLaunchKernelGGL((block_finish_kernel<true, 4>), g, b, 0, s, e, part, splits, M);
    else if (gated)
        hipLaunchKernelGGL((block_finish_kernel<true, 1>), g, b, 0, s, e, part, splits, M);
    else if (wide)
        hipLaunchKernelGGL((block_finish_kernel<false, 4>), g, b, 0, s, e, part, splits, M);
    else
        hipLaunchKernelGGL((block_finish_kernel<false, 1>), g, b, 0, s, e, part, splits, M);
    return launch_status();
}

}  // namespace wqh
