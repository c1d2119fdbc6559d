// The block's forward products for small batches (M <= 32).
//
// y = epilogue(x . W^T) is bound by the weight stream here (2 M flops per
// half byte of 4-bit codes), so the kernel reads every packed word once,
// decodes it in registers and hands the product to the matrix cores, whose
// 16 (or 2 x 16) rows cover all of x.
//
// One v_mfma_f32_16x16x32_f16 takes 16 rows of x and 16 weight rows over 32
// channels: lane l supplies row l % 16 of both, 8 consecutive channels of its
// quarter l / 16.  A lane's weights come as whole chunks (32 codes, 16 bytes
// at 4 bits): chunk 4 t + l / 16 of a row, whose four 8-code blocks feed four
// instructions.  x is read with the same channel mapping, straight from
// global memory: it is small and stays in L2, and nothing has to be staged
// before the stream starts.
//
// A block's eight wavefronts share each output tile (16 weight rows; gated:
// 16 gate rows and the 16 up rows of the same columns, which meet in the
// epilogue of the same thread) and deal its 256-channel steps among them, so
// a wavefront reads whole 128-byte lines and even one tile keeps eight of
// them streaming.  The next step's loads go out before the current one is
// decoded, across tile borders too.  At the end of a tile the eight partial
// products meet in LDS in a fixed order (two buffers: one barrier per tile).
#include <algorithm>

#include "wq_block_common.h"

namespace {

using namespace wq;

constexpr int kWaves = 8;

struct SmallArgs {
    const uint16_t* x;
    const uint32_t* packed;
    const uint16_t* scales;
    const uint8_t* zeros;
    float* part;
    int M, rows, K;
    GroupDiv gd;
    int tiles, sps;
    Epilogue e;
};

// T: 16-row weight tiles per step (gated: 2, the gate's and the up's).
template <int BITS, bool HAS_Z, int MF, int T, bool GATED, bool PART>
__global__ void __launch_bounds__(64 * kWaves) block_small_kernel(const SmallArgs p) {
    static_assert(!GATED || T == 2, "gate and up tiles");
    __shared__ float red[2][kWaves][T * MF][256];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int li = lane & 15, lg = lane >> 4;
    const int chunks = p.K / 32;
    const int G = chunk_group(chunks - 1, p.gd) + 1;
    const int steps = (chunks + 7) / 8;
    // this block's steps of K (blockIdx.y) and this wavefront's among them
    const int s_begin = int(blockIdx.y) * p.sps;
    const int s_end = min(s_begin + p.sps, steps);
    const int mine = (s_end - s_begin - wave + kWaves - 1) / kWaves;  // may be <= 0
    const int half = p.rows / 2;

    struct Regs {
        uint32_t w[T][2][BITS], s[T][2], z[T][2];
        u4 x[2][4][MF];
    };
    // Loads of step st of tile t.  Rows past the matrix and chunks past K
    // read the last ones (their x is zeroed, their outputs are not stored).
    auto load = [&](Regs& r, int t, int st) {
        const int c0 = 8 * st + lg;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = min(c0 + 4 * h, chunks - 1);
            const int g = chunk_group(c, p.gd);
#pragma unroll
            for (int j = 0; j < T; ++j) {
                int n;
                if constexpr (GATED)
                    n = min(16 * t + li, half - 1) + j * half;
                else
                    n = min(16 * (T * t + j) + li, p.rows - 1);
                load_chunk_b<BITS>(p.packed + (size_t(n) * chunks + c) * BITS, r.w[j][h]);
                r.s[j][h] = p.scales[size_t(n) * G + g];
                if constexpr (HAS_Z)
                    r.z[j][h] = p.zeros[size_t(n) * G + g];
                else
                    r.z[j][h] = 1u << (BITS - 1);
            }
#pragma unroll
            for (int f = 0; f < MF; ++f) {
                const u4* xp = reinterpret_cast<const u4*>(p.x + size_t(min(li + 16 * f, p.M - 1)) * p.K + 32 * c);
#pragma unroll
                for (int q = 0; q < 4; ++q) r.x[h][q][f] = xp[q];
            }
        }
    };

    f4 acc[T][MF];
    auto clear = [&]() {
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
            for (int f = 0; f < MF; ++f) acc[j][f] = f4{0.f, 0.f, 0.f, 0.f};
    };
    auto multiply = [&](const Regs& r, int st) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = 8 * st + 4 * h + lg < chunks;
            uint32_t zz[T], ss[T];
#pragma unroll
            for (int j = 0; j < T; ++j) {
                zz[j] = zero_pair_nat<BITS>(r.z[j][h]);
                ss[j] = scale_pair(uint16_t(r.s[j][h]));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                h8 b[T];
#pragma unroll
                for (int j = 0; j < T; ++j) {
                    uint32_t hq[4], v[4];
                    decode_nat<BITS>(r.w[j][h], q, hq);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = as_u32(dequant_pair(hq[i], zz[j], ss[j]));
                    b[j] = __builtin_bit_cast(h8, (u4{v[0], v[1], v[2], v[3]}));
                }
#pragma unroll
                for (int f = 0; f < MF; ++f) {
                    const u4 xv = in ? r.x[h][q][f] : u4{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < T; ++j)
                        acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, xv), b[j], acc[j][f],
                                                                           0, 0, 0);
                }
            }
        }
    };

    // the tile's partial products meet: lane l holds rows 4 (l / 16) + r of
    // column l % 16
    auto tile_end = [&](int t, int parity) {
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
            for (int f = 0; f < MF; ++f)
                *reinterpret_cast<f4*>(&red[parity][wave][j * MF + f][lane * 4]) = acc[j][f];
        __syncthreads();
        constexpr int OT = GATED ? 1 : T;  // output tiles
        for (int o = threadIdx.x; o < p.M * 16 * OT; o += 64 * kWaves) {
            const int nn = o & 15, j = OT == 1 ? 0 : (o >> 4) & (OT - 1), m = o / (16 * OT);
            const int f = m >> 4, at = (16 * ((m & 15) >> 2) + nn) * 4 + (m & 3);
            float a[1] = {0.f}, u[1] = {0.f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                a[0] += red[parity][w][j * MF + f][at];
                if constexpr (GATED) u[0] += red[parity][w][MF + f][at];
            }
            const int col = 16 * (OT * t + j) + nn;
            if constexpr (PART) {
                float* dst = p.part + (size_t(blockIdx.y) * p.M + m) * p.rows;
                if constexpr (GATED) {
                    if (col < half) {
                        dst[col] = a[0];
                        dst[half + col] = u[0];
                    }
                } else if (col < p.rows) {
                    dst[col] = a[0];
                }
            } else {
                if (col < p.e.out) finish<GATED, 1>(p.e, m, col, a, u);
            }
        }
    };

    const int my_tiles = (p.tiles - int(blockIdx.x) + int(gridDim.x) - 1) / int(gridDim.x);
    clear();
    if (mine > 0) {
        const int items = my_tiles * mine;
        int lt = blockIdx.x, lj = 0;  // load cursor: tile, step ordinal
        auto next_load = [&](Regs& r) {
            load(r, lt, s_begin + wave + kWaves * lj);
            if (++lj == mine) {
                lj = 0;
                lt = min(lt + int(gridDim.x), p.tiles - 1);
            }
        };
        Regs cur, nxt;
        next_load(cur);
        int ct = blockIdx.x, cj = 0, k = 0;
        for (int i = 0; i < items; ++i) {
            next_load(nxt);  // past the last item: an in-range re-read
            multiply(cur, s_begin + wave + kWaves * cj);
            if (++cj == mine) {
                cj = 0;
                tile_end(ct, k & 1);
                clear();
                ct += gridDim.x;
                ++k;
            }
            cur = nxt;
        }
    } else {  // no step of its own: this wavefront still meets every barrier
        for (int k = 0; k < my_tiles; ++k) tile_end(int(blockIdx.x) + k * int(gridDim.x), k & 1);
    }
}

struct SmallPlan {
    int T = 1, tiles = 0, blocks = 0, splits = 1, sps = 0;
};

// Launch shape: one wave of resident blocks (two per compute unit), K split
// across blocks where the tiles alone leave most of them without work.
SmallPlan small_plan(int M, int rows, int K, bool gated, size_t part_bytes) {
    SmallPlan p;
    const int cus = wqh::gemm_slots(1);
    const int steps = (K / 32 + 7) / 8;
    p.sps = steps;
    p.T = gated ? 2 : 1;
    p.tiles = gated ? (rows / 2 + 15) / 16 : (rows + 16 * p.T - 1) / (16 * p.T);
    const int slots = 2 * cus;
    while (p.tiles * (p.splits + 1) <= slots && steps >= 2 * kWaves * (p.splits + 1) &&
           size_t(p.splits + 1) * M * rows * 4 <= part_bytes)
        ++p.splits;
    p.sps = (steps + p.splits - 1) / p.splits;
    p.splits = (steps + p.sps - 1) / p.sps;
    p.blocks = std::min(p.tiles, std::max(1, slots / p.splits));
    return p;
}

template <int BITS, bool HAS_Z, int MF>
void launch_small(const wqh::BlockFwd& f, const SmallPlan& pl, const SmallArgs& a, hipStream_t s) {
    const dim3 grid(pl.blocks, pl.splits), block(64 * kWaves);
    if (f.gated) {
        if (pl.splits > 1)
            hipLaunchKernelGGL((block_small_kernel<BITS, HAS_Z, MF, 2, true, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((block_small_kernel<BITS, HAS_Z, MF, 2, true, false>), grid, block, 0, s, a);
    } else {
        if (pl.splits > 1)
            hipLaunchKernelGGL((block_small_kernel<BITS, HAS_Z, MF, 1, false, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((block_small_kernel<BITS, HAS_Z, MF, 1, false, false>), grid, block, 0, s, a);
    }
}

template <int BITS>
void launch_small_bits(const wqh::BlockFwd& f, const SmallPlan& pl, const SmallArgs& a, hipStream_t s) {
    if (f.zeros)
        f.M <= 16 ? launch_small<BITS, true, 1>(f, pl, a, s) : launch_small<BITS, true, 2>(f, pl, a, s);
    else
        f.M <= 16 ? launch_small<BITS, false, 1>(f, pl, a, s) : launch_small<BITS, false, 2>(f, pl, a, s);
}

}  // namespace

namespace wqh {

size_t block_small_part_bytes(int M, int rows, int K, bool gated) {
    const SmallPlan p = small_plan(M, rows, K, gated, ~size_t(0) >> 1);
    return p.splits > 1 ? size_t(p.splits) * M * rows * 4 : 0;
}

wq_status block_small(const BlockFwd& f, float* part, size_t part_bytes, hipStream_t s) {
    const SmallPlan pl = small_plan(f.M, f.rows, f.K, f.gated, part ? part_bytes : 0);
    const SmallArgs a{f.x, f.packed, f.scales, f.zeros, part, f.M, f.rows, f.K, group_magic(f.gs), pl.tiles, pl.sps, f.e};
    switch (f.bits) {
        case 2: launch_small_bits<2>(f, pl, a, s); break;
        case 3: launch_small_bits<3>(f, pl, a, s); break;
        case 4: launch_small_bits<4>(f, pl, a, s); break;
        default: launch_small_bits<8>(f, pl, a, s); break;
    }
    const wq_status st = launch_status();
    if (st != WQ_OK || pl.splits == 1) return st;
    return block_finish(f.e, f.gated, part, pl.splits, f.M, s);
}

}  // namespace wqh
