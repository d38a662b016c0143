// k_fp8_gemm.hip -- block-scaled FP8 products of many rows: dense, and the
// routed experts' gate/up (with SwiGLU and the quantisation of h) and down.
//
//   y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{j in block b} xq[m, j] wq[n, j]
//
// One matrix instruction covers a whole 128-long block, so each block's sum
// starts from zero and enters the fp32 accumulator by one fma with the
// product of its two scales.  The accumulators therefore live in vector
// registers, and the fma's (4 per matrix instruction of 32 cycles) run in the
// shadow of the matrix pipe.
//
// Two forms of a block's sum:
//  - v_mfma_f32_16x16x128_f8f6f4, the full FP8 rate.  It first adds runs of
//    eight products and drops there what lies 13 bits or more below the
//    largest (measured: 1 + 2^-14 in one run gives 1, in two runs 1 + 2^-14;
//    the smaller v_mfma_f32_16x16x32_fp8_fp8 gives the same bits), 1.4e-5
//    relative on random data, but as much as the result where products cancel.
//    Used where the output is rounded to 16 bits and the caller has not asked
//    for fp32 sums (MOE_ACC_F32).
//  - EX: both operands as fp16 (exactly) on v_mfma_f32_16x16x32_f16, half the
//    rate, errors of fp32 sums.  Used for fp32 outputs, with MOE_ACC_F32, and
//    for gate/up, whose result is quantised again: an error of 1e-5 there sends 1 element of 2000
//    to a neighbouring code (measured: the experts' error against 64 bits goes
//    from 3e-4 to 1.1e-3).
//
// fp8_tile_kernel: eight waves own 64*MF rows x 256 weight rows, as RG groups of
// rows x 8 / RG groups of weight rows.  Both operands'
// blocks travel to LDS by direct-to-LDS loads, 8 lanes per 128-byte row block,
// into a ring of two or three stages: one barrier per block, and a block has
// the whole work of another to arrive.  (Read straight into registers in the
// matrix instruction's layout, consecutive lanes are consecutive rows, and the
// L1 then serves 16 bytes a cycle instead of 64: measured 4 times slower.)  A
// wave holds its row fragments of the block and walks its weight
// fragments; each sum enters its accumulator by one fma two sums later.  The
// fma's run in the shadow of the matrix pipe.
//
// Measured (2048 columns of K): 4096 x 11264 with fp16 outputs 105 us (1.8
// PFLOP/s), with fp32 sums (MOE_ACC_F32) 172, with fp32 outputs 175 (1.08);
// experts of 2048 x 1024, top-8 of 64, 4096 tokens: gate/up 279 us, down 110
// (kernels in a run of 60 passes; 340 and 122 in the first ones after a pause),
// the call 390, with fp32 sums in down 434.
// Bounded by instruction issue and by what one workgroup a compute unit exposes:
// of gate/up's 607 k cycles a SIMD the matrix pipe is busy 266 k, other vector
// instructions (half of them conversions) take 271 k, and waves wait 31% of
// theirs; of the product's 228 k 90 k and 78 k, waiting 34%; of down's 257 k 67 k
// and 65 k, waiting 49%.  Moving the loads, the priorities or the conversions
// about changes the time by less than 2%.
//
// gate/up: the 256 weight rows are 128 gate rows and the same 128 up rows (a
// wave holds as many of each), so a workgroup forms 128 columns of h, exactly
// one scale block: h's largest magnitudes meet in LDS, h is quantised with a
// power-of-two scale and leaves as e4m3.
#include <algorithm>
#include <type_traits>

#include "k_fp8_frag.h"

namespace moe {

constexpr int F8_NXCD = 8;
// Dense items go through F8_GROUP row tiles before the next column tile: the
// tiles in flight on an XCD (one per compute unit, 32) then make a patch of
// 4 x 8, whose rows and weights together stay in its L2.  4096 x 11264 x 2048,
// cold: 117 us, against 122 in groups of 8 and 131 through all 16 row tiles.
constexpr int F8_GROUP = 4;

// The work item of a workgroup: column tile nt of row tile mt.  Workgroup i
// runs on XCD i % 8; each XCD takes a contiguous run of items, so that the
// tiles that share weights or rows share an L2.
struct F8Item {
    int mt, nt;
};
template <int MODE>
__device__ __forceinline__ bool f8_item(int MT, int NT, F8Item &it)
{
    const int total = MT * NT;
    const int run = (total + F8_NXCD - 1) / F8_NXCD;
    const int li = blockIdx.x / F8_NXCD;
    const int item = (int)(blockIdx.x % F8_NXCD) * run + li;
    if (li >= run || item >= total)
        return false;
    if constexpr (MODE == F8_DENSE) {
        const int g = item / (F8_GROUP * NT), r = item - g * F8_GROUP * NT;
        const int gm = min(F8_GROUP, MT - g * F8_GROUP);
        it.mt = g * F8_GROUP + r % gm;
        it.nt = r / gm;
    } else {
        it.mt = item / NT;
        it.nt = item % NT;
    }
    return true;
}

// Rows and weights of a row tile; false: nothing to do.
struct F8Tile {
    int row0, rows;
    const uint8_t *w0, *w1;
    const float *s0, *s1;
};
template <int MODE, int BM>
__device__ __forceinline__ bool f8_tile(const Fp8Args &a, int mt, F8Tile &t)
{
    t.w0 = t.w1 = a.w;
    t.s0 = t.s1 = a.ws;
    if constexpr (MODE == F8_DENSE) {
        t.row0 = mt * BM;
        t.rows = min(BM, a.M - t.row0);
    } else {
        const Fp8TileRec r = a.tiles[1 + mt];
        const uint8_t *blob = r.blob;
        if (!blob)
            return false;
        t.row0 = r.row0;
        t.rows = r.rows;
        t.w0 = blob + a.off_w0;
        t.w1 = blob + a.off_w1;
        t.s0 = reinterpret_cast<const float *>(blob + a.off_s0);
        t.s1 = reinterpret_cast<const float *>(blob + a.off_s1);
    }
    return true;
}

// Source row of a tile's row r (rows past the end repeat the last one).
template <int MODE>
__device__ __forceinline__ int64_t f8_xrow(const Fp8Args &a, const F8Tile &t, int r)
{
    const int p = t.row0 + min(r, t.rows - 1);
    return MODE == F8_GATEUP ? a.perm[p] / a.k : p;
}

// Bytes of the last block past K count as zeros on the rows' side (the
// weights' side holds bytes of the same weight row there).
__device__ __forceinline__ int8_8 f8_cut(int8_8 x, int kb, int q, int K)
{
    const int c = kb * 128 + q * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = c < K ? x[i] : 0;
        x[4 + i] = c + 64 < K ? x[4 + i] : 0;
    }
    return x;
}

constexpr int F8_SCW = 8;   // blocks of row scales in LDS at a time (two windows)

template <int MF>
constexpr int f8_stages() { return MF >= 3 ? 2 : 3; }
// The eight waves as groups of rows x groups of weight rows.  A wave converts
// and reads 4 MF / RG row and 2 RG weight fragments for 8 MF sums: 6, 8, 11 and
// 12 of them for MF = 1, 2, 3, 4 (with four groups of rows 9, 10, 11, 12); 6 + 4
// for MF = 3 would be one less, in more registers than there are.  One group for
// MF = 1 is six as well, and 2% slower (256 tokens of 512 experts 82 us against
// 80, four groups 84).
template <int MF>
constexpr int f8_row_groups() { return MF >= 3 ? 4 : 2; }
template <int MF>
constexpr int f8_stage_bytes() { return (64 * MF + 256) * 128; }
// LDS: the ring, two windows of row scales, the weight scales; gate/up's h
// tile and maxima take the ring's place afterwards.
template <int MF>
constexpr int f8_lds(int nkb)
{
    return f8_stages<MF>() * f8_stage_bytes<MF>() + 2 * F8_SCW * 64 * MF * 4 + 2 * nkb * 4;
}

// ES: bytes of an output element (gate/up: not used).
template <int MODE, int MF, bool EX, int ES>
__global__ __launch_bounds__(512, 1) void fp8_tile_kernel(Fp8Args a)
{
    constexpr int NTH = 512;
    constexpr int BM = 64 * MF;
    constexpr int NS = f8_stages<MF>();
    constexpr int STAGE = f8_stage_bytes<MF>();
    constexpr int XB = BM * 128;
    constexpr int PX = MF, PW = 4;   // 16-byte loads per thread and stage
    constexpr int RG = f8_row_groups<MF>(), CG = 8 / RG;   // of the eight waves
    constexpr int XF = 4 * MF / RG, WF = 16 / CG;   // a wave's row and weight fragments
    constexpr int WH = WF / 2;                      // gate/up: of each matrix
    static_assert(PX * 16 * NTH == XB && PW * 16 * NTH == 256 * 128, "whole loads");
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // row fragment m: rows m0 + 16 RG m
    const int m0 = wave / CG * 16, wn = wave % CG;
    const int col = lane & 15, q = lane >> 4;
    const int K = a.K, nkb = (K + 127) / 128;

    const int NT = MODE == F8_GATEUP ? (a.N + 127) / 128 : (a.N + 255) / 256;
    const int MT = MODE == F8_DENSE ? (a.M + BM - 1) / BM : a.tiles[0].rows;
    F8Item it;
    F8Tile t;
    if (!f8_item<MODE>(MT, NT, it) || !f8_tile<MODE, BM>(a, it.mt, t))
        return;
    const int64_t ldw = MODE == F8_DENSE ? a.ldw : K;
    // first column: of h (gate/up), of the output
    const int n0 = it.nt * (MODE == F8_GATEUP ? 128 : 256);

    // Load i of a wave covers 8 rows; lane L fills slot L % 8 of its row, with
    // piece (L % 8) ^ f(row), f(r) = (r >> 1) & 7: the 16 rows of a fragment
    // read hit distinct banks.
    const int lr = wave * 8 + (lane >> 3);            // its row within 64
    const int pc = ((lane & 7) ^ ((lr >> 1) & 7)) * 16;   // 64 divides f's period
    // Rows as indexes and 32-bit offsets from the tile's first weight row
    // (256 ldw < 2^32): the registers are short.
    int xr[PX];
    unsigned wo[PW];
    const uint8_t *wb0 = t.w0 + (int64_t)n0 * ldw, *wb1 = t.w1 + (int64_t)n0 * ldw;
#pragma unroll
    for (int i = 0; i < PX; ++i)
        xr[i] = (int)f8_xrow<MODE>(a, t, i * 64 + lr);
#pragma unroll
    for (int i = 0; i < PW; ++i) {   // gate/up: rows 0..127 gate, 128..255 up
        const int r = MODE == F8_GATEUP ? (i & 1) * 64 + lr : i * 64 + lr;
        wo[i] = (unsigned)min(r, a.N - 1 - n0) * (unsigned)ldw;
    }
    // load i of block kb's PX + PW (past the end re-reads the last block)
    auto issue1 = [&](int kb, int i) {
        uint8_t *st = smem + (kb % NS) * STAGE + wave * 1024;
        const int at = min(min(kb, nkb - 1) * 128 + pc, K - 16);
        if (i < PX)
            dma16(a.x + xr[i < PX ? i : 0] * a.ldx + at, st + i * 8192);
        else
            dma16((MODE == F8_GATEUP && i - PX >= 2 ? wb1 : wb0) +
                      (wo[i < PX ? 0 : i - PX] + (unsigned)at),
                  st + XB + (i - PX) * 8192);
    };
    auto issue = [&](int kb) {
#pragma unroll
        for (int i = 0; i < PX + PW; ++i)
            issue1(kb, i);
    };
    float *xsc = reinterpret_cast<float *>(smem + NS * STAGE);   // [2][F8_SCW][BM]
    float *wsc = xsc + 2 * F8_SCW * BM;                          // [2][nkb]
    // window v of the row scales, transposed; thread t's MF values all in flight
    static_assert(BM * F8_SCW == MF * NTH, "MF scales per thread and window");
    auto scales = [&](int v) {
        float c[MF];
#pragma unroll
        for (int i = 0; i < MF; ++i)
            c[i] = a.xs[f8_xrow<MODE>(a, t, (i * NTH + tid) / F8_SCW) * nkb +
                        min(v * F8_SCW + tid % F8_SCW, nkb - 1)];
#pragma unroll
        for (int i = 0; i < MF; ++i)
            xsc[((v & 1) * F8_SCW + tid % F8_SCW) * BM + (i * NTH + tid) / F8_SCW] = c[i];
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i)
        issue(i);
    scales(0);
    scales(1);
    {
        // the two 128-row scale blocks (gate/up: one of each matrix)
        const float *s1 = MODE == F8_GATEUP ? t.s1 + (int64_t)(n0 >> 7) * nkb
                                            : t.s0 + (int64_t)min((n0 >> 7) + 1, (a.N - 1) >> 7) * nkb;
        const float *s0 = t.s0 + (int64_t)(n0 >> 7) * nkb;
        for (int i = tid; i < 2 * nkb; i += NTH)
            wsc[i] = i < nkb ? s0[i] : s1[i - nkb];
    }

    float4_t acc[XF][WF];
#pragma unroll
    for (int m = 0; m < XF; ++m)
#pragma unroll
        for (int f = 0; f < WF; ++f)
            acc[m][f] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const int sw = (col >> 1) & 7;
    const int o0 = (q ^ sw) * 16, o1 = ((q + 4) ^ sw) * 16;
    // LDS row of weight fragment f: gate/up waves take as many of each matrix
    auto wrow = [&](int f) {
        return (MODE == F8_GATEUP ? f / WH * 128 + wn * (WH * 16) + f % WH * 16
                                  : wn * (WF * 16) + f * 16) + col;
    };
    // MA: the wave's row fragments that hold a row of the tile
    auto block = [&](int kb, auto tail, auto ma) {
        constexpr int MA = decltype(ma)::value;
        // this wave's loads of block kb have landed (those of the NS - 2
        // blocks after it may be pending); after the barrier everyone's have,
        // and the stage of block kb - 1 is read by all
        wait_vm<(NS - 2) * (PX + PW)>();
        lds_barrier();
        if (kb && kb % F8_SCW == 0 && (kb / F8_SCW + 1) * F8_SCW < nkb)
            scales(kb / F8_SCW + 1);   // the window before this one is read by all
        if constexpr (MA == 0) {
            issue(kb + NS - 1);
            return;
        } else {
        const uint8_t *st = smem + (kb % NS) * STAGE;
        auto frag = [&](const uint8_t *r) {
            return join16(*reinterpret_cast<const int4_t *>(r + o0),
                          *reinterpret_cast<const int4_t *>(r + o1));
        };
        // in the order of use, so that the first sum waits for the first reads
        // only
        constexpr int LF = std::min(4, WF);
        constexpr int WD = EX && MF == 4 ? 1 : 2;   // weight fragments read ahead
        constexpr bool WC = EX && WD == 2;          // and converted one ahead
        int8_8 x[MA], w[WD + 1];
        half32 xh[MA];
        float sc[MA][2];
        const float *xs = xsc + (kb & (2 * F8_SCW - 1)) * BM + m0 + col;
        w[0] = frag(st + XB + wrow(0) * 128);
#pragma unroll
        for (int m = 0; m < MA; ++m) {
            x[m] = frag(st + (m * 16 * RG + m0 + col) * 128);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (WD == 2)
            w[1] = frag(st + XB + wrow(1) * 128);
        const float wg = wsc[MODE == F8_GATEUP ? kb : wn * 2 / CG * nkb + kb];
        const float wu = MODE == F8_GATEUP ? wsc[nkb + kb] : wg;
        float xv[MA];
#pragma unroll
        for (int m = 0; m < MA; ++m)
            xv[m] = xs[m * 16 * RG];
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(tail)::value) {
#pragma unroll
            for (int m = 0; m < MA; ++m)
                x[m] = f8_cut(x[m], kb, q, K);
        }
        half32 wh[WC ? 2 : 1];
        float4_t s[4];
        auto add1 = [&](int i, int j) {
            const int f = i / MA, m = i % MA;
            acc[m][f][j] = __builtin_fmaf(s[i & 3][j], sc[m][f / WH], acc[m][f][j]);
        };
        auto add = [&](int i) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                add1(i, j);
        };
#pragma unroll
        for (int f = 0; f < WF; ++f) {
            if (f + WD < WF)
                w[(f + WD) % (WD + 1)] = frag(st + XB + wrow(f + WD) * 128);
            // the next block's loads go out over several fragments: all at once
            // they would hold every wave until the address unit had taken them
#pragma unroll
            for (int i = 0; i < PX + PW; ++i)
                if (i * LF / (PX + PW) == f)
                    issue1(kb + NS - 1, i);
            if constexpr (EX) {
                if (!WC || f == 0)
                    wh[WC ? f & 1 : 0] = f8_to_f16(w[f % (WD + 1)]);
                if (f == 0)
                    xh[0] = f8_to_f16(x[0]);
            }
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int m = 0; m < MA; ++m) {
                const int i = f * MA + m;
                if (f == 0) {
                    sc[m][0] = xv[m] * wg;
                    sc[m][1] = MODE == F8_GATEUP ? xv[m] * wu : sc[m][0];
                }
                if constexpr (EX) {
                    // three vector instructions fit behind each of the four
                    // matrix instructions of a sum: an earlier sum's scaling
                    // and the conversions of the fragments that come next
                    s[i & 3] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i & 3] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            wh[WC ? f & 1 : 0].v[j], xh[m].v[j], s[i & 3], 0, 0, 0);
                        if (i >= 2)
                            add1(i - 2, j);
                        if (f == 0 && m + 1 < MA)
#pragma unroll
                            for (int u = 4 * j; u < 4 * j + 4; ++u)
                                f8_pair(xh[m + 1 < MA ? m + 1 : 0], x[m + 1 < MA ? m + 1 : 0], u);
                        if constexpr (WC)
                            if (f + 1 < WF)
#pragma unroll
                                for (int u = (4 * m + j) * 4 / MA; u < (4 * m + j + 1) * 4 / MA; ++u)
                                    f8_pair(wh[(f + 1) & 1], w[(f + 1) % (WD + 1)], u);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } else {
                    s[i & 3] = mfma_f8(w[f % (WD + 1)], x[m]);
                    if (i >= 2)
                        add(i - 2);
                    // keeps the steps in order: left to itself the scheduler
                    // hoists reads and sums until the registers run out
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            __builtin_amdgcn_s_setprio(0);
        }
        add(WF * MA - 2);
        add(WF * MA - 1);
        }
    };
    auto blocks = [&](auto ma) {
        for (int kb = 0; kb + 1 < nkb; ++kb)
            block(kb, std::false_type(), ma);
        block(nkb - 1, std::true_type(), ma);
    };
    // A short tile's fragments are dealt out over the row groups, and each takes
    // the loop of as many as it has: an expert's last tile costs what it holds
    // (rounded up to 16 RG rows), not its full height.
    const int act = t.rows > m0 ? min(XF, (t.rows - m0 + 16 * RG - 1) / (16 * RG)) : 0;
    if (act == XF)
        blocks(std::integral_constant<int, XF>());
    else if (XF > 3 && act == 3)
        blocks(std::integral_constant<int, std::min(XF, 3)>());
    else if (act == 2)
        blocks(std::integral_constant<int, 2>());
    else if (act == 1)
        blocks(std::integral_constant<int, 1>());
    else
        blocks(std::integral_constant<int, 0>());
    wait_vm<0>();   // trailing loads into LDS are done before it is reused

    if constexpr (MODE == F8_GATEUP) {
        uint8_t *ht = smem;                                              // [BM][128]
        float *mx = reinterpret_cast<float *>(smem + (size_t)BM * 128);   // [CG][BM]
        __syncthreads();   // the ring is read by all
        const bool in = n0 + wn * (WH * 16) < a.N;   // I is a multiple of 64: a wave is in or out
#pragma unroll
        for (int m = 0; m < XF; ++m) {
            float top = 0.0f;
#pragma unroll
            for (int f = 0; f < WH; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float h = in ? swiglu_fast(acc[m][f][i], acc[m][WH + f][i]) : 0.0f;
                    acc[m][f][i] = h;
                    top = fmaxf(top, fabsf(h));
                }
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            if (q == 0)
                mx[wn * BM + m * 16 * RG + m0 + col] = top;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < XF; ++m) {
            const int r = m * 16 * RG + m0 + col;
            float top = mx[r];
#pragma unroll
            for (int i = 1; i < CG; ++i)
                top = fmaxf(top, mx[i * BM + r]);
            const float sc = fp8_scale(top, true), inv = fp8_inv_pow2(sc);
#pragma unroll
            for (int f = 0; f < WH; ++f)
                *reinterpret_cast<int *>(ht + r * 128 + wn * (WH * 16) + f * 16 + q * 4) =
                    fp8_pack4(acc[m][f][0] * inv, acc[m][f][1] * inv, acc[m][f][2] * inv,
                              acc[m][f][3] * inv);
            if (wn == 0 && q == 0 && r < t.rows)
                a.hs[(int64_t)(t.row0 + r) * NT + it.nt] = sc;
        }
        __syncthreads();
        for (int i = tid; i < BM * 8; i += NTH) {
            const int r = i >> 3, c = (i & 7) * 16;
            if (r < t.rows && n0 + c < a.N)
                *reinterpret_cast<int4_t *>(static_cast<uint8_t *>(a.out) +
                                            (int64_t)(t.row0 + r) * a.N + n0 + c) =
                    *reinterpret_cast<const int4_t *>(ht + r * 128 + c);
        }
    } else {
        // through LDS, so that rows leave in whole lines (a lane holds four
        // columns of a row: stored from there, 16 rows by 32 bytes at a time,
        // the 4096 x 11264 product spent a quarter of its time on them)
        const int dt = MODE == F8_DOWN ? MOE_DTYPE_F16 : a.odt;
        constexpr int LR = 256 * ES + 16;            // LDS row, off the banks' period
        constexpr int PASS = ES == 4 && MF > 2 ? (MF == 4 ? 2 : 3) : 1;   // parts of the row fragments that fit
        constexpr int gp = 16 / ES;                  // columns of a 16-byte piece
        const bool vec = (a.ldo * ES) % 16 == 0 && ((uintptr_t)a.out & 15) == 0;
#pragma unroll
        for (int h = 0; h < PASS; ++h) {
            constexpr int MH = XF / PASS;
            __syncthreads();   // the ring, or the first half, is read by all
#pragma unroll
            for (int mm = 0; mm < MH; ++mm) {
                const int m = h * MH + mm;
                const int r = mm * 16 * RG + m0 + col;
#pragma unroll
                for (int f = 0; f < WF; ++f)
                    store4(smem + r * LR, dt, wn * (WF * 16) + f * 16 + q * 4, acc[m][f], 4, true);
            }
            __syncthreads();
            constexpr int np = 256 / gp;   // pieces of a row
            for (int i = tid; i < 16 * RG * MH * np; i += NTH) {
                const int lr2 = i / np, c = (i % np) * gp;
                const int r = h * 16 * RG * MH + lr2;
                const int n = n0 + c;
                if (r >= t.rows || n >= a.N)
                    continue;
                uint8_t *to = static_cast<uint8_t *>(a.out) + ((t.row0 + r) * a.ldo + n) * ES;
                const uint8_t *from = smem + lr2 * LR + c * ES;
                if (vec && n + gp <= a.N) {
                    *reinterpret_cast<int4_t *>(to) = *reinterpret_cast<const int4_t *>(from);
                } else {
                    for (int j = 0; j < gp && n + j < a.N; ++j) {
                        if constexpr (ES == 4)
                            reinterpret_cast<uint32_t *>(to)[j] =
                                reinterpret_cast<const uint32_t *>(from)[j];
                        else
                            reinterpret_cast<uint16_t *>(to)[j] =
                                reinterpret_cast<const uint16_t *>(from)[j];
                    }
                }
            }
        }
    }
}

static int f8_grid(int64_t items, unsigned *grid)
{
    if (items > FP8_MOST_TILES)
        return set_error(MOE_EUNSUPPORTED, "FP8 product: %lld tiles, at most %d",
                         (long long)items, FP8_MOST_TILES);
    *grid = (unsigned)((items + F8_NXCD - 1) / F8_NXCD * F8_NXCD);
    return MOE_OK;
}

template <int MODE, int MF, bool EX, int ES>
static int launch_tile(const Fp8Args &a, int64_t items, hipStream_t s)
{
    static LdsLimit limit;
    unsigned grid;
    int rc = f8_grid(items, &grid);
    if (!rc)
        rc = limit.raise((const void *)fp8_tile_kernel<MODE, MF, EX, ES>, 160 * 1024);
    if (rc)
        return rc;
    hipLaunchKernelGGL((fp8_tile_kernel<MODE, MF, EX, ES>), dim3(grid), dim3(512),
                       f8_lds<MF>((a.K + 127) / 128), s, a);
    MOE_LAUNCH_CHECK("fp8_tile_kernel");
    return MOE_OK;
}

template <int MODE, bool EX>
static int launch_tile_mf(const Fp8Args &a, int mf, int64_t items, hipStream_t s)
{
    switch (mf) {
    case 1: return launch_tile<MODE, 1, EX, 2>(a, items, s);
    case 2: return launch_tile<MODE, 2, EX, 2>(a, items, s);
    default: return launch_tile<MODE, 3, EX, 2>(a, items, s);
    }
}

template <int MF>
static int launch_tile_dense(const Fp8Args &a, bool acc32, hipStream_t s)
{
    const int64_t items = (int64_t)((a.M + 64 * MF - 1) / (64 * MF)) * ((a.N + 255) / 256);
    if (a.odt == MOE_DTYPE_F32)
        return launch_tile<F8_DENSE, MF, true, 4>(a, items, s);
    return acc32 ? launch_tile<F8_DENSE, MF, true, 2>(a, items, s)
                 : launch_tile<F8_DENSE, MF, false, 2>(a, items, s);
}

int launch_fp8_tile_dense(const Fp8Args &a, int mf, bool acc32, hipStream_t s)
{
    switch (mf) {
    case 1: return launch_tile_dense<1>(a, acc32, s);
    case 2: return launch_tile_dense<2>(a, acc32, s);
    case 3: return launch_tile_dense<3>(a, acc32, s);
    default: return launch_tile_dense<4>(a, acc32, s);
    }
}

// Rows of a row tile, 64, 128 or 192, from the mean rows of an expert; fewer
// where that leaves under half the compute units a tile.  Measured (us, H =
// 2048; 64 / 128 / 192 rows): 64 experts of I = 1024, top-8, at 64 tokens 88 /
// 92 / 103, at 256: 95 / 99 / 112, at 512: 121 / 107 / 120, at 1024: 208 /
// 171 / 141, at 4096: 572 / 440 / 378; 60 of I = 1408, top-4, at 512 (34 rows
// an expert): 121 / 125 / 147; 8 of I = 1024, top-2, at 256: 39 / 45 / 47, at
// 1024: 73 / 54 / 63, at 4096: 170 / 148 / 123.  (256-row tiles lost
// everywhere: the registers of the fp16 form do not suffice.)
int fp8_pick_rows(int64_t rows, int E, int I)
{
    const int64_t avg = rows / std::max<int64_t>(1, std::min<int64_t>(E, rows));
    int bm = avg <= 48 ? 64 : avg <= 96 ? 128 : 192;
    while (bm > 64 && (rows + bm - 1) / bm * ((I + 127) / 128) < 128)
        bm -= 64;
    return bm;
}

// Upper bound of row tiles: every expert adds at most one partial tile.
int64_t fp8_tile_bound(int64_t rows, int E, int bm)
{
    return (rows + bm - 1) / bm + std::min<int64_t>(E, rows);
}

// Workgroups of the larger of the routed experts' two launches.
int64_t fp8_most_tiles(int64_t rows, int H, int I, int E)
{
    return fp8_tile_bound(rows, E, fp8_pick_rows(rows, E, I)) *
           std::max((I + 127) / 128, (H + 255) / 256);
}

// Routed experts over the tile table: gate/up into hq/hs, then down into y.
int launch_fp8_experts(Fp8Args a, int bm, uint8_t *hq, float *hs, int H, int I,
                       const int64_t off[6], void *y, bool acc32, hipStream_t s)
{
    const int64_t bound = fp8_tile_bound((int64_t)a.T * a.k, a.E, bm);
    a.ldx = H;
    a.N = I;
    a.K = H;
    a.out = hq;
    a.hs = hs;
    a.off_w0 = off[0];
    a.off_w1 = off[1];
    a.off_s0 = off[3];
    a.off_s1 = off[4];
    int64_t items = bound * ((I + 127) / 128);
    const int rc = launch_tile_mf<F8_GATEUP, true>(a, bm / 64, items, s);
    if (rc)
        return rc;
    a.x = hq;
    a.xs = hs;
    a.ldx = I;
    a.N = H;
    a.K = I;
    a.out = y;
    a.ldo = H;
    a.off_w0 = off[2];
    a.off_s0 = off[5];
    items = bound * ((H + 255) / 256);
    return acc32 ? launch_tile_mf<F8_DOWN, true>(a, bm / 64, items, s)
                 : launch_tile_mf<F8_DOWN, false>(a, bm / 64, items, s);
}

}  // namespace moe
