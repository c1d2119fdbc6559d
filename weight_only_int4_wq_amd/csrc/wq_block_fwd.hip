// The block's forward products for more rows than a decode batch:
// epilogue(x . W^T) on 32x32x16 fp16 matrix-core instructions.
//
// A 256-thread block owns BM x 256 weight rows' worth of products; its four
// wavefronts sit side by side along the weight rows, BM x 64 each, so that
// every weight is decoded by one wavefront only, and the vector work of
// decoding is spread over BM / 32 matrix instructions per fragment.  K
// advances in stages of 64.
//
//  - Weights: lane l supplies 8 consecutive channels (half l / 32 of the
//    stage's 64) of one weight row, which is one packed 8-code block.  A lane
//    loads its own 32-code chunk, scale and zero-point per stage and column
//    block one stage ahead and dequantizes in registers straight into the B
//    operand: decoded weights touch neither LDS nor memory.
//  - The lane's two weight rows are neighbours (2c, 2c + 1) in the linear
//    layer, and gate row o with up row o + I in the gated block: both
//    factors of an output then sit in the same lane's accumulators.
//  - Activations: the BM x 64 tile goes through registers into one of two
//    LDS buffers, a stage ahead; 16-byte unit u of row r at u ^ (r mod 8), so
//    the eight rows that a fragment read takes at a time fall on all banks.
//  - Epilogue: accumulators cross LDS (the activation buffers, free by then)
//    in passes of 32 or 64 rows, so that bias, activation, product, residual
//    and every store work on 8 neighbouring columns (16-byte accesses).
//  - Tiles are dealt to the XCDs in contiguous ranges (tile_coords).
#include <algorithm>

#include "wq_block_common.h"

namespace {

using namespace wq;

struct FwdArgs {
    const uint16_t* x;
    const uint32_t* packed;
    const uint16_t* scales;
    const uint8_t* zeros;
    float* part;
    int M, rows, K;
    GroupDiv gd;
    int m_tiles, n_tiles, tiles, sps;
    Epilogue e;
};

template <int BITS, bool HAS_Z, int BM, bool GATED, bool PART>
__global__ void __launch_bounds__(256, BM == 256 ? 1 : 2) block_fwd_kernel(const FwdArgs p) {
    constexpr int BN = 256, BK = 64, TM = BM / 32, TN = 2;
    constexpr int OC = GATED ? BN / 2 : BN;  // output columns of the tile
    constexpr int ROW = BK * 2;              // bytes of an activation row in LDS
    constexpr int AU = BM * 8 / 256;         // 16-byte units per thread and stage
    constexpr int PASS = BM == 256 ? 64 : 32;
    constexpr int LDS = 2 * BM * ROW > PASS * BN * 4 ? 2 * BM * ROW : PASS * BN * 4;
    __shared__ __attribute__((aligned(128))) uint8_t lds[LDS];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 31, hh = lane >> 5;
    int m_t, n_t;
    tile_coords<4>(blockIdx.x, p.tiles, p.m_tiles, p.n_tiles, m_t, n_t);
    const int m0 = m_t * BM, o0 = n_t * OC;
    const int chunks = p.K / 32;
    const int G = chunk_group(chunks - 1, p.gd) + 1;
    const int stages = (p.K + BK - 1) / BK;
    const int st_begin = int(blockIdx.y) * p.sps;
    const int st_end = min(st_begin + p.sps, stages);

    // ---- activations: thread t copies unit t % 8 of rows t / 8 + 32 i (rows
    // past M read the last one; their outputs are not stored)
    const int au = tid & 7, ar = tid >> 3;
    uint32_t a_off[AU];
#pragma unroll
    for (int i = 0; i < AU; ++i) a_off[i] = uint32_t(min(m0 + ar + 32 * i, p.M - 1) - m0) * uint32_t(p.K) * 2u;
    const char* xbase = reinterpret_cast<const char*>(p.x + size_t(m0) * p.K);
    u4 av[AU];
    auto load_a = [&](int st) {
        const uint32_t k = min(uint32_t(st * BK + 8 * au), uint32_t(p.K - 8)) * 2u;
#pragma unroll
        for (int i = 0; i < AU; ++i) av[i] = *reinterpret_cast<const u4*>(xbase + (a_off[i] + k));
    };
    auto store_a = [&](int st, uint8_t* buf) {
        if (st * BK + 8 * au >= p.K) {  // only in a last stage that K ends in
#pragma unroll
            for (int i = 0; i < AU; ++i) av[i] = u4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int i = 0; i < AU; ++i)
            *reinterpret_cast<u4*>(buf + (ar + 32 * i) * ROW + ((au ^ (ar & 7)) * 16)) = av[i];
    };

    // ---- weights
    const uint32_t* wrow[TN];
    const uint16_t* srow[TN];
    const uint8_t* zrow[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        size_t n;
        if constexpr (GATED)
            n = size_t(min(o0 + wave * 32 + c, p.e.out - 1)) + size_t(j) * p.e.out;
        else
            n = size_t(min(o0 + wave * 64 + 2 * c + j, p.rows - 1));
        wrow[j] = p.packed + n * chunks * BITS;
        srow[j] = p.scales + n * G;
        zrow[j] = HAS_Z ? p.zeros + n * G : nullptr;
    }
    struct BRegs {
        uint32_t w[TN][BITS], s[TN], z[TN];
    };
    auto load_b = [&](BRegs& b, int st) {
        const int cg = min(2 * st + hh, chunks - 1);  // past K: x is zero there
        const int g = chunk_group(cg, p.gd);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            load_chunk_b<BITS>(wrow[j] + cg * BITS, b.w[j]);
            b.s[j] = srow[j][g];
            if constexpr (HAS_Z)
                b.z[j] = zrow[j][g];
            else
                b.z[j] = 1u << (BITS - 1);
        }
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    const uint32_t a_lane = uint32_t(c) * ROW;
    BRegs cur, nxt;
    load_a(st_begin);
    load_b(cur, st_begin);
    store_a(st_begin, lds);
    load_a(min(st_begin + 1, st_end - 1));
    __syncthreads();
    for (int st = st_begin; st < st_end; ++st) {
        const int par = (st - st_begin) & 1;
        const uint8_t* buf = lds + par * (BM * ROW);
        load_b(nxt, min(st + 1, st_end - 1));
        store_a(min(st + 1, st_end - 1), lds + (par ^ 1) * (BM * ROW));
        load_a(min(st + 2, st_end - 1));
        uint32_t zz[TN], ss[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            zz[j] = zero_pair_nat<BITS>(cur.z[j]);
            ss[j] = scale_pair(uint16_t(cur.s[j]));
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            h8 af[TM], bf[TN];
            const uint8_t* ap = buf + a_lane + ((uint32_t(4 * hh + t) ^ uint32_t(c & 7)) * 16u);
#pragma unroll
            for (int i = 0; i < TM; ++i) af[i] = *reinterpret_cast<const h8*>(ap + i * 32 * ROW);
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                uint32_t hq[4], v[4];
                decode_nat<BITS>(cur.w[j], t, hq);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = as_u32(dequant_pair(hq[i], zz[j], ss[j]));
                bf[j] = __builtin_bit_cast(h8, (u4{v[0], v[1], v[2], v[3]}));
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[i], bf[j], acc[i][j], 0, 0, 0);
        }
        cur = nxt;
        __syncthreads();
    }

    // ---- acc[i][j][r]: row 32 i + 8 (r / 4) + 4 hh + r % 4, the lane's j-th
    // weight row
    if constexpr (PART) {
        float* pr = p.part + size_t(blockIdx.y) * p.M * p.rows;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = m0 + 32 * i + 8 * (r >> 2) + 4 * hh + (r & 3);
                const int col = GATED ? o0 + wave * 32 + c : o0 + wave * 64 + 2 * c;
                if (row < p.M) {
                    float* dst = pr + size_t(row) * p.rows;
                    if constexpr (GATED) {
                        if (col < p.e.out) {
                            dst[col] = acc[i][0][r];
                            dst[p.e.out + col] = acc[i][1][r];
                        }
                    } else {
                        if (col < p.rows) dst[col] = acc[i][0][r];
                        if (col + 1 < p.rows) dst[col + 1] = acc[i][1][r];
                    }
                }
            }
    } else {
        float* tile = reinterpret_cast<float*>(lds);  // [PASS][BN]
        const bool wide = p.e.out % 8 == 0;
#pragma unroll
        for (int ps = 0; ps < BM / PASS; ++ps) {
            if (ps) __syncthreads();
#pragma unroll
            for (int ii = 0; ii < PASS / 32; ++ii) {
                const int i = ps * (PASS / 32) + ii;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float* dst = tile + (32 * ii + 8 * (r >> 2) + 4 * hh + (r & 3)) * BN;
                    if constexpr (GATED) {
                        dst[wave * 32 + c] = acc[i][0][r];
                        dst[OC + wave * 32 + c] = acc[i][1][r];
                    } else {
                        *reinterpret_cast<float2*>(dst + wave * 64 + 2 * c) = float2{acc[i][0][r], acc[i][1][r]};
                    }
                }
            }
            __syncthreads();
            constexpr int PER_ROW = OC / 8;
#pragma unroll 1
            for (int q = tid; q < PASS * PER_ROW; q += 256) {
                const int rr = q / PER_ROW, oc = (q % PER_ROW) * 8;
                const int row = m0 + ps * PASS + rr, col = o0 + oc;
                if (row >= p.M || col >= p.e.out) continue;
                const float* src = tile + rr * BN + oc;
                float a[8], u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] = src[i];
                    u[i] = GATED ? src[OC + i] : 0.f;
                }
                if (wide) {
                    finish<GATED, 8>(p.e, row, col, a, u);
                } else {
#pragma unroll 1
                    for (int i = 0; i < 8 && col + i < p.e.out; ++i) {
                        float a1[1] = {src[i]}, u1[1] = {GATED ? src[OC + i] : 0.f};
                        finish<GATED, 1>(p.e, row, col + i, a1, u1);
                    }
                }
            }
        }
    }
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

struct FwdPlan {
    int BM = 128, splits = 1, sps = 0;
};

// Tile height and K split by a time model: a tile takes a fixed time per
// 64-deep stage (the larger of its matrix instructions and its weight
// stream), tiles run in rounds of the resident blocks, a split writes and
// re-reads fp32 partial sums.
FwdPlan fwd_plan(int M, int rows, int K, int bits, bool gated, size_t part_bytes) {
    const int cus = wqh::gemm_slots(1);
    const int stages = (K + 63) / 64;
    const int n_tiles = gated ? (rows / 2 + 127) / 128 : (rows + 255) / 256;
    FwdPlan best;
    best.sps = stages;
    double best_us = 1e30;
    const int heights[3] = {64, 128, 256};
    for (int h = 0; h < 3; ++h) {
        const int BM = heights[h];
        const double stage_us = BM == 64 ? 0.45 : BM == 128 ? 0.75 : 1.2;
        const int slots = cus * (BM == 256 ? 1 : 2);
        const double share = BM == 256 ? 1.0 : 2.0;  // resident blocks share the unit
        const long long tiles = (long long)((M + BM - 1) / BM) * n_tiles;
        for (int S = 1; S <= 32; ++S) {
            const int sps = (stages + S - 1) / S;
            const int Se = (stages + sps - 1) / sps;
            if (Se != S) continue;
            if (S > 1 && (sps < 4 || double(Se) * M * rows * 4.0 > double(part_bytes))) break;
            const long long blocks = tiles * Se;
            const double rounds = double((blocks + slots - 1) / slots);
            const double fill = blocks < cus ? 1.0 : share;  // one block per unit runs alone
            double us = rounds * sps * stage_us * (blocks <= cus ? 0.6 : 1.0) * fill / share;
            if (blocks <= cus) us = sps * stage_us * 0.6;
            us += 3.0;
            if (S > 1) us += 2.0 + double(Se) * M * rows * 8.0 / 4e6;
            if (us < best_us * 0.98) {
                best_us = us;
                best.BM = BM;
                best.splits = Se;
                best.sps = sps;
            }
        }
    }
    (void)bits;
    return best;
}

template <int BITS, bool HAS_Z, int BM>
void launch_fwd(const wqh::BlockFwd& f, const FwdPlan& pl, const FwdArgs& a, hipStream_t s) {
    const dim3 grid(a.tiles, pl.splits), block(256);
    if (f.gated) {
        if (pl.splits > 1)
            hipLaunchKernelGGL((block_fwd_kernel<BITS, HAS_Z, BM, true, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((block_fwd_kernel<BITS, HAS_Z, BM, true, false>), grid, block, 0, s, a);
    } else {
        if (pl.splits > 1)
            hipLaunchKernelGGL((block_fwd_kernel<BITS, HAS_Z, BM, false, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((block_fwd_kernel<BITS, HAS_Z, BM, false, false>), grid, block, 0, s, a);
    }
}

template <int BITS, bool HAS_Z>
void launch_fwd_bm(const wqh::BlockFwd& f, const FwdPlan& pl, const FwdArgs& a, hipStream_t s) {
    switch (pl.BM) {
        case 64: launch_fwd<BITS, HAS_Z, 64>(f, pl, a, s); break;
        case 128: launch_fwd<BITS, HAS_Z, 128>(f, pl, a, s); break;
        default: launch_fwd<BITS, HAS_Z, 256>(f, pl, a, s); break;
    }
}

template <int BITS>
void launch_fwd_bits(const wqh::BlockFwd& f, const FwdPlan& pl, const FwdArgs& a, hipStream_t s) {
    f.zeros ? launch_fwd_bm<BITS, true>(f, pl, a, s) : launch_fwd_bm<BITS, false>(f, pl, a, s);
}

}  // namespace

namespace wqh {

size_t block_fwd_part_bytes(int M, int rows, int K, int bits, bool gated) {
    const FwdPlan p = fwd_plan(M, rows, K, bits, gated, ~size_t(0) >> 1);
    return p.splits > 1 ? size_t(p.splits) * M * rows * 4 : 0;
}

wq_status block_fwd(const BlockFwd& f, float* part, size_t part_bytes, hipStream_t s) {
    const FwdPlan pl = fwd_plan(f.M, f.rows, f.K, f.bits, f.gated, part ? part_bytes : 0);
    const int oc = f.gated ? 128 : 256;
    const int m_tiles = (f.M + pl.BM - 1) / pl.BM, n_tiles = (f.e.out + oc - 1) / oc;
    const FwdArgs a{f.x,    f.packed,           f.scales, f.zeros, part,    f.M, f.rows,
                    f.K,    group_magic(f.gs),  m_tiles,  n_tiles, m_tiles * n_tiles, pl.sps, f.e};
    switch (f.bits) {
        case 2: launch_fwd_bits<2>(f, pl, a, s); break;
        case 3: launch_fwd_bits<3>(f, pl, a, s); break;
        case 4: launch_fwd_bits<4>(f, pl, a, s); break;
        default: launch_fwd_bits<8>(f, pl, a, s); break;
    }
    const wq_status st = launch_status();
    if (st != WQ_OK || pl.splits == 1) return st;
    return block_finish(f.e, f.gated, part, pl.splits, f.M, s);
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
