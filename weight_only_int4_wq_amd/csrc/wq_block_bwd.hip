// The block's backward pass: dz from the incoming gradient and the kept
// pre-activations, dx = dz . W (+ dx_add), dbias = column sums of dz.
//
// dx [M][K] = dz [M][R] . W [R][K] sums over the weight rows, while the codes
// are packed along K.  The matrix instruction wants 8 consecutive n of one
// column per lane; a packed word holds 8 columns of one n.  So a lane takes
// the same 8-code block of 8 consecutive weight rows and turns the 8 x 8
// square while decoding, at no cost: the byte permutes that expose two codes
// of one row in the forward decoder here pick one byte of two neighbouring
// rows, and the pair's two scales and zero-points differ instead of being
// equal.  (At 4 bits: one permute per two pairs, one and-or per pair, one
// subtraction and one multiplication: exactly the forward weights.)
//
// Since every lane holds 8 columns, a wavefront decodes 256 columns x 16 rows
// at once, too many to keep for itself: the block (BM x 256 outputs, 64
// weight rows a stage) decodes each stage once, a quarter per wavefront, into
// LDS in the order the fragments are read (1 KB per fragment, no bank
// conflicts either way), and its 2 x 2 wavefronts, BM/2 x 128 outputs each,
// read it from there: every weight is decoded once per block, not once per
// wavefront that multiplies it.
// The columns are dealt to fragments so that a lane ends up with 4
// consecutive outputs of a row: one 8-byte store (16 bytes of partial sums).
//
// Stages overlap in one loop with one barrier: while stage s is multiplied
// from its LDS buffers, stage s + 1 is decoded into the others and stage
// s + 2 is loaded into registers; scales and zero-points (64 rows x the
// tile's groups) pass through LDS one stage earlier.  Tiles that would fill a
// last round only partly are cut along the weight rows.
//
// dz enters the product in fp16, the matrix instruction's operand: half a step
// (2^-11) of each value, which puts as much error into dx as dx's own rounding
// does (relative to dx, root mean square: 2.1e-4 each, 2.9e-4 together), and an
// infinity past 65504, which takes its row of dx along.  Two operands (the
// value and what its rounding left) would take twice the matrix instructions.
//
// Measured: dz [2048 x 4096] . W [4096 x 11008] at 4 bits 198 us a pass (934
// TFLOP/s), of which the cut tiles' sums take 10; [2048 x 22016] . [22016 x
// 4096] 348 us (1063 TFLOP/s) of its pass's 401, and 17 for its sums.  Bound by
// the matrix units at the clock that power leaves them (busy 51 % of the counted
// cycles) and by the LDS writes of the decoded weights, which hold a wavefront
// up by 25 cycles each.
#include <algorithm>

#include "wq_block_common.h"

namespace {

using namespace wq;

// ------------------------------------------------------------------ dz ----

struct DzArgs {
    const uint16_t* dy;      // [M][N]
    const uint16_t* preact;  // [M][R], null for WQ_ACT_NONE (linear only)
    uint16_t* dz;            // [M][R], nullable
    uint16_t* dzp;           // [M][ld], zero past R, nullable
    float* dbias;            // [gridDim.y][R] sums of this row range, nullable
    int M, N, R, ld, act, rows_per;
};

constexpr int kDzRowLanes = 4;  // rows a block works on at once

// A block takes 64 V-wide column groups and rows_per rows, four at a time;
// dbias's sums stay in registers, cross the four row lanes through LDS and
// leave as one partial row per block row.  V = 8 needs N to be a multiple of
// 8.  Bound by memory: each of dy, preact and dz is touched once (gated, 2048
// x 11008, 225 MB in 45 us).  Columns that are not 8-byte groups take V = 1,
// bound by the activation's arithmetic (311 x 5001, gelu, 7.1 us).
template <bool GATED, int V>
__global__ void __launch_bounds__(64 * kDzRowLanes) block_dz_kernel(const DzArgs p) {
    constexpr int P = GATED ? 2 : 1;
    __shared__ float red[kDzRowLanes][P][64 * V];
    const int cl = threadIdx.x & 63, rl = threadIdx.x >> 6;
    const int col = (int(blockIdx.x) * 64 + cl) * V;
    const int r0 = int(blockIdx.y) * p.rows_per, r1 = min(r0 + p.rows_per, p.M);
    float sum[P][V];
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[q][i] = 0.f;
    for (int m = r0 + rl; m < r1; m += kDzRowLanes) {
        if (col < p.N) {
            float d[V], z[P][V], o[P][V];
            load_h<V>(p.dy + size_t(m) * p.N + col, d);
            if (p.preact) {
#pragma unroll
                for (int q = 0; q < P; ++q) load_h<V>(p.preact + size_t(m) * p.R + q * p.N + col, z[q]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) z[0][i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float a;
                const float s = act_slope(z[0][i], p.act, a);
                if constexpr (GATED) {
                    o[0][i] = d[i] * z[1][i] * s;
                    o[1][i] = d[i] * a;
                } else {
                    o[0][i] = d[i] * s;
                }
            }
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const int n = q * p.N + col;
                if (p.dz) store_h<V>(p.dz + size_t(m) * p.R + n, o[q]);
                if (p.dzp) {
#pragma unroll
                    for (int i = 0; i < V; ++i) p.dzp[size_t(m) * p.ld + n + i] = f2h(o[q][i]);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) sum[q][i] += o[q][i];
            }
        }
        // the padding of dzp's rows (fewer than 8 columns)
        if (p.dzp && blockIdx.x == 0 && cl < p.ld - p.R) p.dzp[size_t(m) * p.ld + p.R + cl] = 0;
    }
    if (!p.dbias) return;
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) red[rl][q][i * 64 + cl] = sum[q][i];
    __syncthreads();
    for (int t = threadIdx.x; t < P * 64 * V; t += 64 * kDzRowLanes) {
        const int q = t / (64 * V), at = t - q * 64 * V;
        const int c = (int(blockIdx.x) * 64 + (at & 63)) * V + (at >> 6);
        if (c >= p.N) continue;
        float v = red[0][q][at];
#pragma unroll
        for (int l = 1; l < kDzRowLanes; ++l) v += red[l][q][at];
        p.dbias[size_t(blockIdx.y) * p.R + q * p.N + c] = v;
    }
}

// out[i] = sum over the row ranges, in order; zero for none.
__global__ void __launch_bounds__(256) block_dbias_kernel(const float* __restrict__ part, int ranges, int R,
                                                          float* __restrict__ out) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= R) return;
    float v = 0.f;
    int r = 0;
    for (; r + 8 <= ranges; r += 8) {  // (eight loads in flight)
        float w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = part[size_t(r + k) * R + i];
#pragma unroll
        for (int k = 0; k < 8; ++k) v += w[k];
    }
    for (; r < ranges; ++r) v += part[size_t(r) * R + i];
    out[i] = v;
}

// ------------------------------------------------------------------ dx ----

// Vector instructions issued after each matrix instruction.
#ifndef WQ_BLOCK_DX_VALU
#define WQ_BLOCK_DX_VALU 4
#endif

struct DxArgs {
    const uint16_t* dz;  // [M][ld], ld a multiple of 8, zero from R to ld
    const uint32_t* packed;
    const uint16_t* scales;
    const uint8_t* zeros;
    const uint16_t* add;  // [M][K], nullable, may be dx
    uint16_t* dx;
    float* part;  // [ranges][tail tiles][BM][256] partial products
    int M, R, K, ld;
    GroupDiv gd;
    int m_tiles, k_tiles, tiles, head, sps;
};

// One weight row's 8-code block: 8 * BITS bits in the low bits of w[0] (w[1]
// above for 8-bit codes).  `blk` is the row's block index.
template <int BITS>
struct RowBlock {
    static constexpr int kWords = BITS == 8 ? 2 : 1;
};
template <int BITS>
__device__ __forceinline__ void load_row_block(const char* row, uint32_t blk, uint32_t* w) {
    if constexpr (BITS == 4) {
        w[0] = *reinterpret_cast<const uint32_t*>(row + blk * 4u);
    } else if constexpr (BITS == 8) {
        typedef uint32_t u2 __attribute__((ext_vector_type(2)));
        const u2 v = *reinterpret_cast<const u2*>(row + blk * 8u);
        w[0] = v.x;
        w[1] = v.y;
    } else if constexpr (BITS == 2) {
        w[0] = *reinterpret_cast<const uint16_t*>(row + blk * 2u);
    } else {
        // the 3 bytes at byte 3 blk: within one aligned word for blocks 0 and 3
        // of a chunk, across two for blocks 1 and 2 (inside the row either way)
        const uint32_t b = 3u * blk, q = blk & 3u;
        const uint32_t at = (b & ~3u);
        const uint32_t lo = *reinterpret_cast<const uint32_t*>(row + at);
        const uint32_t hi = *reinterpret_cast<const uint32_t*>(row + (q == 1u || q == 2u ? at + 4u : at));
        w[0] = __builtin_amdgcn_alignbyte(hi, lo, b & 3u) & 0x00FFFFFFu;
    }
}

// Columns 2 i and 2 i + 1 of two neighbouring rows' blocks a and b: out[0] and
// out[1] hold the pairs (row of a, row of b) of (q - z) * s, each row with its
// own z and s.
template <int BITS>
__device__ __forceinline__ void decode_columns(int i, const uint32_t* a, const uint32_t* b, uint32_t z, uint32_t ss,
                                               uint32_t (&out)[2]) {
    const uint32_t ze = z | kMagic2;
    if constexpr (BITS == 4) {
        const uint32_t sel = 0x0C000C00u | ((4u + i) << 16) | uint32_t(i);
        const uint32_t t = __builtin_amdgcn_perm(b[0], a[0], sel);
        out[0] = as_u32(dequant_pair(and_or(t, 0x000F000Fu, kMagic2), ze, ss));
        out[1] = as_u32(dequant_pair(and_or(t, 0x00F000F0u, 0x54005400u), (z << 4) | 0x54005400u, ss));
    } else if constexpr (BITS == 8) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t k = uint32_t((2 * i + e) & 3), w = uint32_t(2 * i) >> 2;
            const uint32_t sel = 0x0C000C00u | ((4u + k) << 16) | k;
            out[e] = as_u32(dequant_pair(__builtin_amdgcn_perm(b[w], a[w], sel) | kMagic2, ze, ss));
        }
    } else if constexpr (BITS == 2) {
        const uint32_t t = (a[0] | (b[0] << 16)) >> (4 * i);
        out[0] = as_u32(dequant_pair(and_or(t, 0x00030003u, kMagic2), ze, ss));
        out[1] = as_u32(dequant_pair(and_or(t >> 2, 0x00030003u, kMagic2), ze, ss));
    } else {
        // six bits of each row; what b's half carries above them is masked
        const uint32_t t = ((a[0] >> (6 * i)) & 0x3Fu) | ((b[0] >> (6 * i)) << 16);
        out[0] = as_u32(dequant_pair(and_or(t, 0x00070007u, kMagic2), ze, ss));
        out[1] = as_u32(dequant_pair(and_or(t >> 3, 0x00070007u, kMagic2), ze, ss));
    }
}

// Four columns of one row: dx = fp16(v + add); with perm, column k' of the
// packed order belongs to channel perm[k'].
__device__ __forceinline__ void finish_dx(const uint16_t* add, uint16_t* dx, const int32_t* perm, size_t row_at, int col,
                                          float (&v)[4]) {
    if (perm) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const size_t at = row_at + perm[col + q];
            dx[at] = f2h(v[q] + (add ? h2f(add[at]) : 0.f));
        }
        return;
    }
    if (add) {
        float b[4];
        load_h<4>(add + row_at + col, b);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += b[q];
    }
    store_h<4>(dx + row_at + col, v);
}

// G8: groups of 32 channels, up to 8 groups per tile; otherwise up to 4
// (group sizes of 64 and more, tiles start at multiples of 256).
template <int BITS, int BM, bool G8>
__global__ void __launch_bounds__(256) block_dx_kernel(const DxArgs p) {
    constexpr int BK = 64, TM = BM / 64, TN = 4;
    constexpr int ROW = BK * 2;
    constexpr int AU = BM * 8 / 256;
    constexpr int NG = G8 ? 8 : 4;
    constexpr int A_BYTES = BM * ROW, B_BYTES = 256 * BK * 2, S_BYTES = NG * BK * 2;
    constexpr int W = RowBlock<BITS>::kWords;
    extern __shared__ __attribute__((aligned(128))) uint8_t lds[];
    uint8_t* const lds_a = lds;                        // [2][BM rows][64 n]
    uint8_t* const lds_b = lds_a + 2 * A_BYTES;        // [2][4 k-steps][2][4][64 lanes] x 16 bytes
    uint8_t* const lds_s = lds_b + 2 * B_BYTES;        // [2][NG][64] scales, then zero-points

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int c = lane & 31, hh = lane >> 5;
    const TileWork tw = tile_work(blockIdx.x, p.tiles, p.head, p.m_tiles, p.k_tiles);
    const int m0 = tw.m_t * BM, k0 = tw.n_t * 256;
    const int chunks = p.K / 32;
    const int G = chunk_group(chunks - 1, p.gd) + 1;
    const int stages = (p.R + BK - 1) / BK;
    const int st_begin = tw.split * p.sps;
    const int st_end = tw.part < 0 ? stages : min(st_begin + p.sps, stages);
    const int st_last = st_end - 1;

    // ---- dz: thread t copies unit t % 8 of rows t / 8 + 32 i
    const int au = tid & 7, ar = tid >> 3;
    uint32_t a_off[AU];
#pragma unroll
    for (int i = 0; i < AU; ++i) a_off[i] = uint32_t(min(m0 + ar + 32 * i, p.M - 1) - m0) * uint32_t(p.ld) * 2u;
    const char* abase = reinterpret_cast<const char*>(p.dz + size_t(m0) * p.ld);
    u4 av[AU];
    auto load_a = [&](int st) {
        const uint32_t n = min(uint32_t(st * BK + 8 * au), uint32_t(p.ld - 8)) * 2u;
#pragma unroll
        for (int i = 0; i < AU; ++i) av[i] = *reinterpret_cast<const u4*>(abase + (a_off[i] + n));
    };
    auto store_a = [&](int st, int par) {
        const uint32_t keep = st * BK + 8 * au < p.ld ? ~0u : 0u;  // zeros past R
        uint8_t* buf = lds_a + par * A_BYTES;
#pragma unroll
        for (int i = 0; i < AU; ++i)
            *reinterpret_cast<u4*>(buf + (ar + 32 * i) * ROW + ((au ^ ((ar >> 1) & 7)) * 16)) =
                av[i] & u4{keep, keep, keep, keep};
    };

    // ---- scales and zero-points: thread t takes row t % 64 of groups t / 64
    // (and t / 64 + 4), rows past R with scale 0
    const int g0 = chunk_group(k0 / 32, p.gd);
    const int g_last = chunk_group(min(k0 / 32 + 7, chunks - 1), p.gd);
    const uint8_t* zp = p.zeros ? p.zeros : reinterpret_cast<const uint8_t*>(p.scales);  // always loaded
    uint32_t sv[NG / 4], zv[NG / 4], s_off[NG / 4];
    int s_g[NG / 4];
#pragma unroll
    for (int i = 0; i < NG / 4; ++i) {
        s_g[i] = min(g0 + (tid >> 6) + 4 * i, g_last);
        s_off[i] = uint32_t(tid & 63) * uint32_t(G) + uint32_t(s_g[i]);
    }
    auto load_s = [&](int st) {
        const size_t row0 = size_t(st) * BK * G;
        const uint32_t most = uint32_t(min(p.R - 1 - st * BK, BK - 1)) * uint32_t(G);  // the last row's
#pragma unroll
        for (int i = 0; i < NG / 4; ++i) {
            const uint32_t o = min(s_off[i], most + uint32_t(s_g[i]));
            sv[i] = (p.scales + row0)[o];
            zv[i] = (zp + row0)[o];
        }
    };
    auto store_s = [&](int st, int par) {
        const bool in = st * BK + (tid & 63) < p.R;
        uint16_t* s = reinterpret_cast<uint16_t*>(lds_s + par * 2 * S_BYTES);
#pragma unroll
        for (int i = 0; i < NG / 4; ++i) {
            const int at = ((tid >> 6) + 4 * i) * BK + (tid & 63);
            s[at] = in ? uint16_t(sv[i]) : uint16_t(0);
            s[NG * BK + at] = uint16_t(p.zeros ? zv[i] : 1u << (BITS - 1));
        }
    };

    // ---- weights: this wavefront decodes rows 16 wave + 8 hh + i of the
    // stage, block c of the tile's 32 (blocks past K read the last one; their
    // outputs are not stored)
    const uint32_t blk = uint32_t(min(k0 / 8 + c, p.K / 8 - 1));
    const int lg = chunk_group(int(blk >> 2), p.gd) - g0;
    const size_t row_bytes = size_t(chunks) * BITS * 4;
    uint32_t wv[8][W], wnext[8][W];  // the next stage's words, the one's after
    uint32_t w_off[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w_off[i] = uint32_t(16 * wave + 8 * hh + i) * uint32_t(row_bytes);
    auto load_w = [&](int st, uint32_t (&w)[8][W]) {
        const char* base = reinterpret_cast<const char*>(p.packed) + size_t(st) * BK * row_bytes;
        const uint32_t most = uint32_t(min(p.R - 1 - st * BK, BK - 1)) * uint32_t(row_bytes);  // the last row
#pragma unroll
        for (int i = 0; i < 8; ++i) load_row_block<BITS>(base + min(w_off[i], most), blk, w[i]);
    };
    // Column pairs i0 .. i1 - 1 (of 4) of the wavefront's share, into LDS in
    // the fragments' order.
    auto decode = [&](int par, int i0, int i1) {
        const uint8_t* s = lds_s + par * 2 * S_BYTES + (lg * BK + 16 * wave + 8 * hh) * 2;
        const u4 ss = *reinterpret_cast<const u4*>(s);
        const u4 zz = *reinterpret_cast<const u4*>(s + S_BYTES);
        const uint32_t sa[4] = {ss.x, ss.y, ss.z, ss.w}, za[4] = {zz.x, zz.y, zz.z, zz.w};
        uint8_t* dst = lds_b + par * B_BYTES + ((wave * 2 + (c >> 4)) * 4 * 64 + hh * 32 + (c & 15)) * 16;
#pragma unroll
        for (int i = i0; i < i1; ++i) {
            uint32_t f[4][2];
#pragma unroll
            for (int q = 0; q < 4; ++q) decode_columns<BITS>(i, wv[2 * q], wv[2 * q + 1], za[q], sa[q], f[q]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 2 * i + e;
                *reinterpret_cast<u4*>(dst + ((j & 3) * 64 + (j >> 2) * 16) * 16) =
                    u4{f[0][e], f[1][e], f[2][e], f[3][e]};
            }
        }
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    auto read_ab = [&](int par, int t, h8 (&a)[TM], h8 (&b)[TN]) {
        const uint8_t* ab = lds_a + par * A_BYTES + (wm * (BM / 2) + c) * ROW +
                            ((uint32_t(2 * t + hh) ^ uint32_t((c >> 1) & 7)) * 16u);
        const uint8_t* bb = lds_b + par * B_BYTES + (wn * 4 * 64 + lane) * 16 + t * 8192;
#pragma unroll
        for (int i = 0; i < TM; ++i) a[i] = *reinterpret_cast<const h8*>(ab + i * 32 * ROW);
#pragma unroll
        for (int j = 0; j < TN; ++j) b[j] = *reinterpret_cast<const h8*>(bb + j * 1024);
    };
    auto multiply = [&](const h8 (&a)[TM], const h8 (&b)[TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[i], b[j], acc[i][j], 0, 0, 0);
    };
    constexpr int NM = TM * TN, NR = TM + TN, NV = WQ_BLOCK_DX_VALU;

    load_s(st_begin);
    load_w(st_begin, wv);
    load_a(st_begin);
    store_s(st_begin, 0);
    load_s(min(st_begin + 1, st_last));
    store_s(min(st_begin + 1, st_last), 1);
    __syncthreads();
    decode(0, 0, 4);
    store_a(st_begin, 0);
    // (in the loop's order, so that its waits count the same loads from the
    // first stage on)
    load_w(min(st_begin + 1, st_last), wnext);
    load_s(min(st_begin + 2, st_last));
    load_a(min(st_begin + 1, st_last));
    __syncthreads();
    h8 af[2][TM], bf[2][TN];
    read_ab(0, 0, af[0], bf[0]);
    for (int st = st_begin; st < st_end; ++st) {
        const int par = (st - st_begin) & 1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int w = 0; w < W; ++w) wv[i][w] = wnext[i][w];
        read_ab(par, 1, af[1], bf[1]);
        load_w(min(st + 2, st_last), wnext);
        decode(par ^ 1, 0, 2);  // stage st + 1
        multiply(af[0], bf[0]);
        sched_step<NM, NR + 2, 4, 8, NV>();
        read_ab(par, 2, af[0], bf[0]);
        decode(par ^ 1, 2, 4);
        store_s(min(st + 2, st_last), par);
        load_s(min(st + 3, st_last));
        multiply(af[1], bf[1]);
        sched_step<NM, NR + 2, 4 + NG / 2, NG / 2, NV>();
        read_ab(par, 3, af[1], bf[1]);
        store_a(min(st + 1, st_last), par ^ 1);
        load_a(min(st + 2, st_last));
        multiply(af[0], bf[0]);
        sched_step<NM, NR, AU, AU, NV>();
        __syncthreads();
        read_ab(par ^ 1, 0, af[0], bf[0]);
        multiply(af[1], bf[1]);
        sched_step<NM, NR, 0, 0, NV>();
    }

    // ---- acc[i][j][r]: row 32 i + 8 (r / 4) + 4 hh + r % 4, column
    // 8 (c % 16) + 4 (c / 16) + j of the wavefront's BM/2 x 128
    const int lc = wn * 128 + 8 * (c & 15) + 4 * (c >> 4);
    if (tw.part >= 0) {  // the whole tile, rows and columns past the matrix too
        float* pr = p.part + size_t(tw.part) * (BM * 256) + lc;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int lr = wm * (BM / 2) + 32 * i + 8 * (r >> 2) + 4 * hh + (r & 3);
                *reinterpret_cast<f4*>(pr + lr * 256) = f4{acc[i][0][r], acc[i][1][r], acc[i][2][r], acc[i][3][r]};
                if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // few accumulators on their way at a time
            }
        return;
    }
    const int col = k0 + lc;
    if (col >= p.K) return;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = m0 + wm * (BM / 2) + 32 * i + 8 * (r >> 2) + 4 * hh + (r & 3);
            if (row >= p.M) continue;
            float v[4] = {acc[i][0][r], acc[i][1][r], acc[i][2][r], acc[i][3][r]};
            finish_dx(p.add, p.dx, nullptr, size_t(row) * p.K, col, v);
        }
}

// The same for tiles cut in ranges (with act-order, for every tile): block b
// takes 4 rows of a tail tile, four columns per thread; the ranges' partial
// products are added in order.  A launch's blocks count from `first`.
template <int BM>
__global__ void __launch_bounds__(256) block_dx_tail_kernel(const DxArgs p, int splits,
                                                            const int32_t* __restrict__ perm, int first) {
    const int tail = p.tiles - p.head, b = first + int(blockIdx.x), i = b / (BM / 4);
    int m_t, k_t;
    tile_place(p.head + i, p.m_tiles, p.k_tiles, m_t, k_t);
    const int rr = (b % (BM / 4)) * 4 + threadIdx.x / 64, lc = (threadIdx.x & 63) * 4;
    const int row = m_t * BM + rr, col = k_t * 256 + lc;
    if (row >= p.M || col >= p.K) return;
    const int at[1] = {lc};
    f4 w[1];
    sum_ranges(p.part + (size_t(i) * BM + rr) * 256, at, size_t(tail) * (BM * 256), splits, w);
    float v[4] = {w[0][0], w[0][1], w[0][2], w[0][3]};
    finish_dx(p.add, p.dx, perm, size_t(row) * p.K, col, v);
}

// dx of an empty sum: dx_add, or zero.
__global__ void __launch_bounds__(256) block_dx_empty_kernel(size_t n4, const uint16_t* add, uint16_t* dx) {
    for (size_t i = size_t(blockIdx.x) * 256 + threadIdx.x; i < n4; i += size_t(gridDim.x) * 256) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        finish_dx(add, dx, nullptr, i * 4, 0, v);
    }
}

// [3 bits]: codes that straddle bytes take longer to decode (taller tiles
// decode them fewer times), and the loop waits for all of its loads, its next
// stage's among them, before each decoding.  At 256 rows it also moves 128
// accumulators a stage to make room in registers (8 bits: 96; 2 and 4: none).
constexpr wqh::TileCosts kDxCosts[2] = {
    {{{64, 0.55, 0.36, 8.01, false}, {128, 1.09, 0.14, 6.7, false}, {256, 1.44, 0.48, 6.29, false}}, 0.17, 0.314},
    {{{64, 1.35, 0.29, 0.02, false}, {128, 2.24, 0.17, 0.0, false}, {256, 2.75, 0.0, 0.0, false}}, 7.27, 0.259}};

wqh::TilePlan dx_plan(int M, int R, int K, int bits, bool has_perm, size_t part_bytes) {
    return wqh::plan_tiles(M, (K + 255) / 256, (R + 63) / 64, kDxCosts[bits == 3], 1, part_bytes, wqh::gemm_slots(1),
                           has_perm);
}

template <int BITS, int BM, bool G8>
wq_status launch_dx(const wqh::TilePlan& pl, const int32_t* perm, const DxArgs& a, hipStream_t s) {
    constexpr int lds = 2 * (BM * 128 + 256 * 128 + 2 * (G8 ? 8 : 4) * 128);
    auto kern = block_dx_kernel<BITS, BM, G8>;
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return wqh::hip_status(e);
    hipLaunchKernelGGL(kern, dim3(pl.blocks()), dim3(256), lds, s, a);
    const wq_status st = wqh::launch_status();
    if (st != WQ_OK || pl.tail() == 0) return st;
    return wqh::launch_pieces(pl.tail() * (BM / 4LL), [&](unsigned blocks, int first) {
        hipLaunchKernelGGL((block_dx_tail_kernel<BM>), dim3(blocks), dim3(256), 0, s, a, pl.splits, perm, first);
    });
}

template <int BITS>
wq_status launch_dx_bits(const wqh::TilePlan& pl, const int32_t* perm, bool g8, const DxArgs& a, hipStream_t s) {
    switch (pl.BM) {
        case 64: return g8 ? launch_dx<BITS, 64, true>(pl, perm, a, s) : launch_dx<BITS, 64, false>(pl, perm, a, s);
        case 128: return g8 ? launch_dx<BITS, 128, true>(pl, perm, a, s) : launch_dx<BITS, 128, false>(pl, perm, a, s);
        default: return g8 ? launch_dx<BITS, 256, true>(pl, perm, a, s) : launch_dx<BITS, 256, false>(pl, perm, a, s);
    }
}

size_t round256(size_t b) { return (b + 255) & ~size_t(255); }

// dbias's row ranges: enough blocks to fill the machine, of about 16 rows or
// more (17 rows make two, of 9 and 8; the last takes what is left): a partial
// row costs 4 bytes per column to write and read.
int dbias_ranges(int M, int R) {
    const int col_blocks = (R + 511) / 512;
    const int want = (4 * wqh::gemm_slots(1) + col_blocks - 1) / col_blocks;
    return std::max(1, std::min(want, (M + 15) / 16));
}

struct BwdBytes {
    size_t dz, dbias, dx;  // dx: partial products, act-order's among them
};

BwdBytes bwd_bytes(int M, int R, int K, int bits, bool has_perm) {
    BwdBytes b{};
    b.dz = round256(size_t(M) * ((size_t(R) + 7) / 8 * 8) * 2);
    b.dbias = round256(size_t(dbias_ranges(M, R)) * R * 4);
    b.dx = dx_plan(M, R, K, bits, has_perm, ~size_t(0)).part_bytes();
    return b;
}

}  // namespace

namespace wqh {

size_t block_bwd_workspace_bytes(int M, int R, int K, int bits, bool has_perm) {
    if (M <= 0 || R <= 0) return 0;
    const BwdBytes b = bwd_bytes(M, R, K, bits, has_perm);
    return b.dz + b.dbias + b.dx;
}

wq_status block_bwd(const uint16_t* dy, const uint16_t* preact, int act, bool gated, const uint32_t* packed,
                    const uint16_t* scales, const uint8_t* zeros, const int32_t* perm, const uint16_t* add,
                    uint16_t* dx, uint16_t* dz, float* dbias, int M, int N, int K, int bits, int gs, void* workspace,
                    size_t ws_bytes, hipStream_t s) {
    const int R = gated ? 2 * N : N;
    if (R == 0) {  // an empty sum
        if (M == 0) return WQ_OK;
        const size_t n4 = size_t(M) * (K / 4);
        hipLaunchKernelGGL(block_dx_empty_kernel, dim3(unsigned(std::min<size_t>((n4 + 255) / 256, gemm_slots(8)))),
                           dim3(256), 0, s, n4, add, dx);
        return launch_status();
    }
    if (M == 0) {
        if (!dbias) return WQ_OK;
        hipLaunchKernelGGL(block_dbias_kernel, dim3((R + 255) / 256), dim3(256), 0, s, nullptr, 0, R, dbias);
        return launch_status();
    }
    // ---- workspace: [dz][dbias partial sums][fp32 dx]
    const bool none = act == WQ_ACT_NONE && !gated;
    const bool aligned = R % 8 == 0;
    const int ld = (R + 7) / 8 * 8;
    const bool own_dz = !aligned || (!none && !dz);
    const int ranges = dbias ? dbias_ranges(M, R) : 0;
    char* w = static_cast<char*>(workspace);
    size_t left = workspace ? ws_bytes : 0;
    auto take = [&](size_t bytes) -> char* {
        bytes = round256(bytes);
        if (bytes > left) return nullptr;
        char* r = w;
        w += bytes;
        left -= bytes;
        return r;
    };
    uint16_t* dzp = nullptr;
    float* dbp = nullptr;
    if (own_dz && !(dzp = reinterpret_cast<uint16_t*>(take(size_t(M) * ld * 2)))) return WQ_ERR_ARG;
    const uint16_t* operand = own_dz ? dzp : none ? dy : dz;
    if (own_dz && aligned) {  // no padding: written as dz is
        dz = dzp;
        dzp = nullptr;
    }
    if (ranges > 1 && !(dbp = reinterpret_cast<float*>(take(size_t(ranges) * R * 4)))) return WQ_ERR_ARG;
    const TilePlan pl = dx_plan(M, R, K, bits, perm != nullptr, left);
    if (pl.tiles == 0) return WQ_ERR_ARG;

    // ---- dz, dbias
    if (!none || own_dz || dz || dbias) {
        DzArgs a{dy, none ? nullptr : preact, dz, dzp, ranges > 1 ? dbp : dbias, M, N, R, ld, act, 0};
        // without dbias: short row ranges, for many blocks
        const int per = ranges ? (M + ranges - 1) / ranges
                               : std::max((M + 65534) / 65535, std::max(4, std::min(32, (M + 63) / 64 * 4)));
        a.rows_per = per;
        const int gy = (M + per - 1) / per;
        const bool wide = N % 8 == 0;
        const int cols = 64 * (wide ? 8 : 1);
        const dim3 grid((N + cols - 1) / cols, gy), block(64 * kDzRowLanes);
        if (gated && wide)
            hipLaunchKernelGGL((block_dz_kernel<true, 8>), grid, block, 0, s, a);
        else if (gated)
            hipLaunchKernelGGL((block_dz_kernel<true, 1>), grid, block, 0, s, a);
        else if (wide)
            hipLaunchKernelGGL((block_dz_kernel<false, 8>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((block_dz_kernel<false, 1>), grid, block, 0, s, a);
        wq_status st = launch_status();
        if (st != WQ_OK) return st;
        if (ranges > 1) {
            hipLaunchKernelGGL(block_dbias_kernel, dim3((R + 255) / 256), dim3(256), 0, s, dbp, gy, R, dbias);
            st = launch_status();
            if (st != WQ_OK) return st;
        }
    }

    // ---- dx
    const int m_tiles = (M + pl.BM - 1) / pl.BM, k_tiles = (K + 255) / 256;
    const DxArgs a{operand, packed, scales, zeros, add, dx, reinterpret_cast<float*>(w), M, R, K, ld, group_magic(gs),
                   m_tiles, k_tiles, pl.tiles, pl.head, pl.sps};
    const bool g8 = gs < 64;
    switch (bits) {
        case 2: return launch_dx_bits<2>(pl, perm, g8, a, s);
        case 3: return launch_dx_bits<3>(pl, perm, g8, a, s);
        case 4: return launch_dx_bits<4>(pl, perm, g8, a, s);
        default: return launch_dx_bits<8>(pl, perm, g8, a, s);
    }
}

}  // namespace wqh
