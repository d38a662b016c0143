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
// A workgroup of four waves owns 16*MF rows x 256 weight rows; wave w owns 64
// of the weight rows and reads them straight from memory into registers (no
// other wave needs them, so LDS would only add traffic), one block ahead.
// MF = 8: the rows' blocks pass through a three-stage LDS ring filled by
// direct-to-LDS loads and are shared by the waves.  MF <= 4: few rows, each
// wave loads them itself, and there is no barrier in the loop.
//
// gate/up: the 256 weight rows are 128 gate rows and the same 128 up rows (a
// wave holds 32 + 32), so a workgroup forms 128 columns of h, exactly one
// scale block: h's largest magnitudes meet in LDS, h is quantised with a
// power-of-two scale and leaves as e4m3.
#include <algorithm>

#include "k_fp8_frag.h"

namespace moe {

constexpr int F8_NXCD = 8;

template <int MF>
constexpr int f8_stage() { return MF * 16 * 128; }
// LDS: three stages of rows and their scales (MF = 8), or the epilogue's
// h tile and maxima (gate/up); never both at once.
template <int MODE, int MF, bool EX>
size_t f8_lds(int nkb)
{
    const size_t loop = MF == 8 ? 3 * (size_t)f8_stage<MF>() + (size_t)nkb * MF * 16 * 4 : 0;
    const size_t epi = MODE == F8_GATEUP ? (size_t)MF * 16 * (128 + 16) : 0;
    return loop > epi ? loop : epi;
}

template <int MODE, int MF, bool EX>
__global__ __launch_bounds__(256, MF >= 4 ? 1 : 2) void fp8_tile_kernel(Fp8Args a)
{
    constexpr bool XLDS = MF == 8;
    constexpr int BM = 16 * MF;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, q = lane >> 4;
    const int K = a.K, nkb = (K + 127) / 128;

    // work item: column tile nt of row tile mt.  Workgroup i runs on XCD
    // i % 8; each XCD takes a contiguous run of items.
    const int NT = MODE == F8_GATEUP ? (a.N + 127) / 128 : (a.N + 255) / 256;
    const int MT = MODE == F8_DENSE ? (a.M + BM - 1) / BM : a.tiles[0];
    const int total = MT * NT;
    const int run = (total + F8_NXCD - 1) / F8_NXCD;
    const int li = blockIdx.x / F8_NXCD;
    const int item = (int)(blockIdx.x % F8_NXCD) * run + li;
    if (li >= run || item >= total)
        return;
    const int mt = MODE == F8_DENSE ? item % MT : item / NT;
    const int nt = MODE == F8_DENSE ? item / MT : item % NT;

    int row0, rows;
    const uint8_t *w0 = a.w, *w1 = a.w;
    const float *s0 = a.ws, *s1 = a.ws;
    if constexpr (MODE == F8_DENSE) {
        row0 = mt * BM;
        rows = min(BM, a.M - row0);
    } else {
        const int e = a.tiles[2 + 2 * mt];
        row0 = a.tiles[3 + 2 * mt];
        rows = min(BM, a.offsets[e + 1] - row0);
        const uint8_t *blob = static_cast<const uint8_t *>(a.blobs[e]);
        if (!blob)
            return;
        w0 = blob + a.off_w0;
        w1 = blob + a.off_w1;
        s0 = reinterpret_cast<const float *>(blob + a.off_s0);
        s1 = reinterpret_cast<const float *>(blob + a.off_s1);
    }

    // weights: fragment f of this wave, lane row col
    const int64_t ldw = MODE == F8_DENSE ? a.ldw : K;
    const uint8_t *wr[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        const uint8_t *base;
        int n;
        if constexpr (MODE == F8_GATEUP) {
            base = f < 2 ? w0 : w1;
            n = nt * 128 + wave * 32 + (f & 1) * 16 + col;
        } else {
            base = w0;
            n = nt * 256 + wave * 64 + f * 16 + col;
        }
        wr[f] = base + (int64_t)min(n, a.N - 1) * ldw;
    }
    // the wave's columns lie in one 128-column scale block (two for gate/up:
    // one of each matrix)
    const int sb = MODE == F8_GATEUP ? nt : min(nt * 256 + wave * 64, a.N - 1) >> 7;
    s0 += (int64_t)sb * nkb;
    s1 += (int64_t)sb * nkb;

    // source row of the tile's row r (rows past the end repeat the last one)
    auto xrow = [&](int r) -> int64_t {
        const int p = row0 + min(r, rows - 1);
        return MODE == F8_GATEUP ? a.perm[p] / a.k : p;
    };
    const int klast = K - 16;
    int4_t wf[2][4][2];
    float wsc[2][2];
    auto load_w = [&](int kb, int b) {
        kb = min(kb, nkb - 1);
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                wf[b][f][h] =
                    ldg(reinterpret_cast<const int4_t *>(wr[f] + min(kb * 128 + h * 64 + q * 16, klast)));
        wsc[b][0] = s0[kb];
        wsc[b][1] = MODE == F8_GATEUP ? s1[kb] : 0.0f;
    };

    float4_t acc[MF][4];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int f = 0; f < 4; ++f)
            acc[m][f] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    half32 wh[4];   // EX: the block's weights as fp16
    auto begin = [&](int b) {
        if constexpr (EX) {
#pragma unroll
            for (int f = 0; f < 4; ++f)
                wh[f] = f8_to_f16(join16(wf[b][f][0], wf[b][f][1]));
        }
    };
    auto step = [&](int m, int b, int8_8 xf, float xs) {
        half32 xh;
        if constexpr (EX)
            xh = f8_to_f16(xf);
        const float sg = xs * wsc[b][0];
        const float su = MODE == F8_GATEUP ? xs * wsc[b][1] : sg;
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            float4_t t;
            if constexpr (EX)
                t = mfma_f16(wh[f], xh);
            else
                t = mfma_f8(join16(wf[b][f][0], wf[b][f][1]), xf);
            const float s = f < 2 ? sg : su;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[m][f][i] = __builtin_fmaf(t[i], s, acc[m][f][i]);
        }
    };
    // bytes of the last block past K count as zeros (the weights' side reads
    // bytes of the same row there instead)
    auto cut = [&](int8_8 xf, int kb) {
        const int c = kb * 128 + q * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            xf[i] = c < K ? xf[i] : 0;
            xf[4 + i] = c + 64 < K ? xf[4 + i] : 0;
        }
        return xf;
    };
    const bool ragged = (K & 127) != 0;

    if constexpr (XLDS) {
        constexpr int STAGE = f8_stage<MF>();
        constexpr int PX = STAGE / 4096;   // 16-byte loads per thread per stage
        float *sl = reinterpret_cast<float *>(smem + 3 * STAGE);   // [nkb][BM]
        // load i of wave w covers rows 8 (4 i + w) ..+7; lane L fills slot
        // L % 8 of its row, i.e. piece (L % 8) ^ f(row), f(r) = (r >> 1) & 7:
        // the 16 rows of a fragment read hit distinct banks
        const uint8_t *src[PX];
        int pc[PX];
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int r = (i * 4 + wave) * 8 + (lane >> 3);
            pc[i] = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
            src[i] = a.x + xrow(r) * a.ldx;
        }
        auto issue = [&](int kb) {   // past the end re-reads the last block
            uint8_t *st = smem + (kb % 3) * STAGE;
            kb = min(kb, nkb - 1);
#pragma unroll
            for (int i = 0; i < PX; ++i)
                dma16(src[i] + min(kb * 128 + pc[i], klast), st + (i * 4 + wave) * 1024);
        };
        // rows' scales, transposed
        for (int i = tid; i < BM * nkb; i += 256) {
            const int r = i / nkb, kb = i - r * nkb;
            sl[kb * BM + r] = a.xs[xrow(r) * nkb + kb];
        }
        load_w(0, 0);
        issue(0);
        issue(1);
        const int sw = (col >> 1) & 7;
        const int o0 = (q ^ sw) * 16, o1 = ((q + 4) ^ sw) * 16;
        auto body = [&](int kb, int b) {
            // this wave's weights and row loads of block kb have landed (only
            // the PX row loads of block kb + 1 may be pending); after the
            // barrier everyone's have, and block kb - 1 is read by all
            wait_vm<PX>();
            lds_barrier();
            begin(b);
            load_w(kb + 1, b ^ 1);
            issue(kb + 2);
            const uint8_t *st = smem + (kb % 3) * STAGE;
            const bool tail = ragged && kb == nkb - 1;
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                const uint8_t *r = st + (m * 16 + col) * 128;
                int8_8 xf = join16(*reinterpret_cast<const int4_t *>(r + o0),
                                   *reinterpret_cast<const int4_t *>(r + o1));
                if (tail)
                    xf = cut(xf, kb);
                step(m, b, xf, sl[kb * BM + m * 16 + col]);
            }
        };
        for (int kb = 0; kb < nkb; kb += 2) {
            body(kb, 0);
            if (kb + 1 < nkb)
                body(kb + 1, 1);
        }
        wait_vm<0>();   // trailing loads into LDS are done before it is reused
    } else {
        const uint8_t *xr[MF];
        const float *xsr[MF];
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int64_t r = xrow(m * 16 + col);
            xr[m] = a.x + r * a.ldx;
            xsr[m] = a.xs + r * nkb;
        }
        int4_t xf[2][MF][2];
        float xs[2][MF];
        auto load_x = [&](int kb, int b) {
            kb = min(kb, nkb - 1);
#pragma unroll
            for (int m = 0; m < MF; ++m) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    xf[b][m][h] = ldg(reinterpret_cast<const int4_t *>(
                        xr[m] + min(kb * 128 + h * 64 + q * 16, klast)));
                xs[b][m] = xsr[m][kb];
            }
        };
        auto body = [&](int kb, int b) {
            begin(b);
            load_w(kb + 1, b ^ 1);
            load_x(kb + 1, b ^ 1);
            const bool tail = ragged && kb == nkb - 1;
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                int8_8 v = join16(xf[b][m][0], xf[b][m][1]);
                if (tail)
                    v = cut(v, kb);
                step(m, b, v, xs[b][m]);
            }
        };
        load_w(0, 0);
        load_x(0, 0);
        for (int kb = 0; kb < nkb; kb += 2) {
            body(kb, 0);
            if (kb + 1 < nkb)
                body(kb + 1, 1);
        }
    }

    if constexpr (MODE == F8_GATEUP) {
        uint8_t *ht = smem;                                              // [BM][128]
        float *mx = reinterpret_cast<float *>(smem + (size_t)BM * 128);   // [4][BM]
        __syncthreads();   // the ring is read by all
        const int i0 = nt * 128 + wave * 32;   // I is a multiple of 64: a wave is in or out
        const bool in = i0 < a.N;
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            float top = 0.0f;
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float h = in ? swiglu_fast(acc[m][f][i], acc[m][2 + f][i]) : 0.0f;
                    acc[m][f][i] = h;
                    top = fmaxf(top, fabsf(h));
                }
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            if (q == 0)
                mx[wave * BM + m * 16 + col] = top;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int r = m * 16 + col;
            const float top = fmaxf(fmaxf(mx[r], mx[BM + r]), fmaxf(mx[2 * BM + r], mx[3 * BM + r]));
            const float s = fp8_scale(top, true), inv = fp8_inv_pow2(s);
#pragma unroll
            for (int f = 0; f < 2; ++f)
                *reinterpret_cast<int *>(ht + r * 128 + wave * 32 + f * 16 + q * 4) =
                    fp8_pack4(acc[m][f][0] * inv, acc[m][f][1] * inv, acc[m][f][2] * inv,
                              acc[m][f][3] * inv);
            if (wave == 0 && q == 0 && r < rows)
                a.hs[(int64_t)(row0 + r) * NT + nt] = s;
        }
        __syncthreads();
        for (int i = tid; i < BM * 8; i += 256) {
            const int r = i >> 3, c = (i & 7) * 16;
            if (r < rows && nt * 128 + c < a.N)
                *reinterpret_cast<int4_t *>(static_cast<uint8_t *>(a.out) +
                                            (int64_t)(row0 + r) * a.N + nt * 128 + c) =
                    *reinterpret_cast<const int4_t *>(ht + r * 128 + c);
        }
    } else {
        const int dt = MODE == F8_DOWN ? MOE_DTYPE_F16 : a.odt;
        const bool vec = MODE == F8_DOWN || (a.ldo % 4 == 0 && ((uintptr_t)a.out & 15) == 0);
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int r = m * 16 + col;
            if (r >= rows)
                continue;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int n = nt * 256 + wave * 64 + f * 16 + q * 4;
                if (n < a.N)
                    store4(a.out, dt, (int64_t)(row0 + r) * a.ldo + n, acc[m][f], a.N - n, vec);
            }
        }
    }
}

template <int MODE, int MF, bool EX>
static int launch_tile(const Fp8Args &a, int64_t items, hipStream_t s)
{
    const size_t lds = f8_lds<MODE, MF, EX>((a.K + 127) / 128);
    static bool attr_set = false;   // raising the LDS limit is idempotent
    if (lds > 65536 && !attr_set) {
        MOE_HIP_TRY(hipFuncSetAttribute((const void *)fp8_tile_kernel<MODE, MF, EX>,
                                        hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024));
        attr_set = true;
    }
    const int64_t grid = (items + F8_NXCD - 1) / F8_NXCD * F8_NXCD;
    if (grid > 0x7fffffffLL)
        return set_error(MOE_EUNSUPPORTED, "FP8 product: more than 2^31 - 1 tiles");
    hipLaunchKernelGGL((fp8_tile_kernel<MODE, MF, EX>), dim3((unsigned)grid), dim3(256), lds, s, a);
    MOE_LAUNCH_CHECK("fp8_tile_kernel");
    return MOE_OK;
}

template <int MODE, bool EX>
static int launch_tile_mf(const Fp8Args &a, int mf, int64_t items, hipStream_t s)
{
    switch (mf) {
    case 1: return launch_tile<MODE, 1, EX>(a, items, s);
    case 2: return launch_tile<MODE, 2, EX>(a, items, s);
    case 4: return launch_tile<MODE, 4, EX>(a, items, s);
    default: return launch_tile<MODE, 8, EX>(a, items, s);
    }
}

int launch_fp8_tile_dense(const Fp8Args &a, hipStream_t s)
{
    const int64_t items = (int64_t)((a.M + 127) / 128) * ((a.N + 255) / 256);
    if (a.odt == MOE_DTYPE_F32)
        return launch_tile<F8_DENSE, 8, true>(a, items, s);
    return launch_tile<F8_DENSE, 8, false>(a, items, s);
}

// Row-tile height (16 MF rows) from the mean rows of an expert.
int fp8_pick_mf(int64_t rows, int E)
{
    const int64_t avg = rows / std::max<int64_t>(1, std::min<int64_t>(E, rows));
    return avg <= 12 ? 1 : avg <= 24 ? 2 : avg <= 64 ? 4 : 8;
}

// Upper bound of row tiles: every expert adds at most one partial tile.
int64_t fp8_tile_bound(int64_t rows, int E, int mf)
{
    return (rows + 16 * mf - 1) / (16 * mf) + std::min<int64_t>(E, rows);
}

// Routed experts over the tile table: gate/up into hq/hs, then down into y.
int launch_fp8_experts(Fp8Args a, int mf, uint8_t *hq, float *hs, int H, int I,
                       const int64_t off[6], void *y, hipStream_t s)
{
    const int64_t bound = fp8_tile_bound((int64_t)a.T * a.k, a.E, mf);
    a.ldx = H;
    a.N = I;
    a.K = H;
    a.out = hq;
    a.hs = hs;
    a.off_w0 = off[0];
    a.off_w1 = off[1];
    a.off_s0 = off[3];
    a.off_s1 = off[4];
    const int rc = launch_tile_mf<F8_GATEUP, true>(a, mf, bound * ((I + 127) / 128), s);
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
    return launch_tile_mf<F8_DOWN, false>(a, mf, bound * ((H + 255) / 256), s);
}

}  // namespace moe
