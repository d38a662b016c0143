// k_fp8_decode.hip -- block-scaled FP8 products of few rows: decode tokens
// through the routed experts, and dense products of few rows.
//
//   y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{j in block b} xq[m, j] wq[n, j]
//
// Bound by the weights' stream from memory: each weight byte is used for one
// row tile only, so the kernel's task is to have many bytes in flight.  A
// workgroup owns 32 weight rows (gate/up: 16 gate rows and the same 16 up
// rows, so that it also forms h) and its four waves take every fourth
// 128-long block of K each.  A wave has one block in flight, in a stage of its
// own in LDS filled by direct-to-LDS loads of 8 lanes per 128-byte row block
// (loaded straight into the matrix instruction's layout, consecutive lanes are
// consecutive rows, and the L1 serves 16 bytes a cycle instead of 64).  Several
// workgroups share a compute unit, as many as its LDS (stages, decode rows, 8 KB
// of sums, 16 for 32 rows) and registers hold: gate/up at H = 2048 five with one
// token, four with four, two with sixteen; down at I = 1024 six with one, five
// with four; dense four (16 rows) or three (32).  So many small stages beat few
// deep ones (64 experts, 4 tokens: 31.5 us with one stage per wave, 35 with two,
// 50 with four, at a floor of 30.5; one token 14.7, 15.4, 16.8).  No barrier is
// needed until the waves' sums meet in LDS, in wave order, so that results do not
// depend on timing.  The tokens are the matrix core's second operand, 16 to a
// fragment; its idle columns cost nothing here.  The fp16 form of a block's sum
// (fp32 accuracy).
//
// Measured: 1 x 5632 x 2048 5.1 us a call, 4.1 on the card (11.5 MB, whose loads
// alone need 2.2: a wave's four blocks of K come one after the other), 333 x 1408
// x 2000 with fp32 outputs 6.9 us; experts of 2048 x 1024, top-8 of 64: one token
// 14.3 us for 50 MB (3.5 TB/s), four 32.5 us for 176 MB in 28 experts (part of it
// from the last-level cache in back-to-back calls), eight 47.5 for 258 in 41.
//
// Decode experts quantise their rows in the workgroup (gate/up: the fp16
// tokens; down: the fp32 h the first launch left in the workspace), hidden
// behind the weight loads: no launch of its own.
#include <algorithm>

#include "k_fp8_frag.h"

namespace moe {

// One row's 128-blocks to e4m3 in LDS by 16-lane groups.
template <typename XT>
__device__ __forceinline__ void quant_row_lds(const XT *src, int K, int kb, int c, uint8_t *dst,
                                              float *sc)
{
    float v[8];
    const int at = kb * 128 + c * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = 0.0f;
    if (at < K) {   // K is a multiple of 64: eight values are all in or all out
        if constexpr (sizeof(XT) == 2) {
            const half8_t h = *reinterpret_cast<const half8_t *>(src + at);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = (float)h[i];
        } else {
            const float4_t a = *reinterpret_cast<const float4_t *>(src + at);
            const float4_t b = *reinterpret_cast<const float4_t *>(src + at + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        }
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = fmaxf(m, fabsf(v[i]));
    const float s = fp8_scale(row16_max(m), true);
    const float inv = fp8_inv_pow2(s);
    int2_t q;
    q[0] = fp8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    q[1] = fp8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    *reinterpret_cast<int2_t *>(dst + kb * 128 + c * 8) = q;
    if (c == 0)
        sc[kb] = s;
}

// Bytes of a wave's stage: 32 weight rows, dense also 16 MT token rows, and
// the scales.
template <int MODE, int MT>
constexpr int f8_rows_stage()
{
    return (4 + (MODE == F8_DENSE ? 2 * MT : 0)) * 1024 + 256;
}

// MODE F8_DENSE: grid (32-column tiles, 16*MT-row tiles).  F8_GATEUP /
// F8_DOWN: grid (tiles of 16 intermediate / 32 output columns, sorted rows);
// the workgroups at an expert's first row and every 16th (every T-th) after it
// serve the rows up to the next, the others leave at once.  Nothing is predicated
// between a matrix instruction and the use of its result (on the path that jumps
// over predicated loads the compiler leaves out wait states): rows past the end
// repeat the last one (their columns are not stored), blocks past the end
// repeat the last one with a weight scale of zero.
template <int MODE, int MT>
__global__ __launch_bounds__(256) void fp8_rows_kernel(Fp8Args a)
{
    static_assert(MT == 1 || (MODE == F8_DENSE && MT == 2), "at most 32 rows; experts 16");
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[4][2 * MT][64][4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, q = lane >> 4;
    const int K = a.K, nkb = (K + 127) / 128;

    int row0 = blockIdx.y * 16 * MT, rows = min(16 * MT, a.M - row0);
    const int held = min(a.T, FP8_DECODE_ROWS);   // decode: rows of a workgroup
    const uint8_t *w0 = a.w, *w1 = a.w;
    const float *s0 = a.ws, *s1 = a.ws;
    if constexpr (MODE != F8_DENSE) {
        const int p = blockIdx.y;
        // the expert of sorted row p: the experts that end at or before it;
        // its run's bounds come from the same lanes
        int e = 0, first = 0, end = 0;
        for (int b = 0; b < a.E; b += 64) {
            const int o = b + lane < a.E ? a.offsets[b + lane + 1] : 0x7fffffff;
            const int n = __popcll(__ballot(o <= p));
            if (n)
                first = __builtin_amdgcn_readlane(o, n - 1);
            e += n;
            if (n < 64) {
                end = __builtin_amdgcn_readlane(o, n);
                break;
            }
        }
        if (e >= a.E)
            return;   // behind the last routed row
        if ((p - first) % held)
            return;
        row0 = p;
        rows = min(held, end - p);
        const uint8_t *blob = static_cast<const uint8_t *>(a.blobs[e]);
        if (!blob)
            return;
        w0 = blob + a.off_w0;
        w1 = blob + a.off_w1;
        s0 = reinterpret_cast<const float *>(blob + a.off_s0);
        s1 = reinterpret_cast<const float *>(blob + a.off_s1);
    }
    const int n0 = MODE == F8_GATEUP ? blockIdx.x * 16 : blockIdx.x * 32;
    const int64_t ldw = MODE == F8_DENSE ? a.ldw : K;
    s0 += (int64_t)(n0 >> 7) * nkb;
    s1 += (int64_t)(n0 >> 7) * nkb;   // 32 columns never leave their scale block

    // The wave's stage: 32 weight rows (gate/up: 16 + 16), and dense also the
    // 16 MT token rows, of 128 bytes.  Load i covers rows 8i..8i+7; lane L
    // fills slot L % 8 of its row with piece (L % 8) ^ f(row), f(r) = (r >> 1)
    // & 7, so that the 16 rows of a fragment read hit distinct banks.
    constexpr int XR = MODE == F8_DENSE ? 2 * MT : 0;   // loads of token rows
    // then the block's scales, one lane each: dense rows 0.., from 32 the weights'
    constexpr int STAGE = f8_rows_stage<MODE, MT>();
    uint8_t *const st = smem + wave * STAGE;
    const uint8_t *src[4 + XR];
    int pc[4 + XR];
#pragma unroll
    for (int i = 0; i < 4 + XR; ++i) {
        const int r = (i < 4 ? i : i - 4) * 8 + (lane >> 3);
        pc[i] = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
        if (i >= 4)
            src[i] = a.x + (int64_t)(row0 + min(r, rows - 1)) * a.ldx;
        else if (MODE == F8_GATEUP)
            src[i] = (i < 2 ? w0 : w1) + (int64_t)(n0 + (r & 15)) * ldw;
        else
            src[i] = w0 + (int64_t)min(n0 + r, a.N - 1) * ldw;
    }
    const float *scp = lane == 32 ? s0 : s1;
    if (MODE == F8_DENSE && lane < 16 * MT)
        scp = a.xs + (int64_t)(row0 + min(lane, rows - 1)) * nkb;
    // this wave's block j (past the end the last one again)
    auto block_of = [&](int j) { return min(4 * j + wave, nkb - 1); };
    auto issue = [&](int j) {
        const int at = block_of(j) * 128;
#pragma unroll
        for (int i = 0; i < 4 + XR; ++i)
            dma16(src[i] + min(at + pc[i], K - 16), st + i * 1024);
        dma4(scp + block_of(j), st + (4 + XR) * 1024);
    };
    issue(0);

    float4_t acc[2][MT];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            acc[f][m] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

    uint8_t *xl = smem + 4 * STAGE;                                        // decode: [held][nkb*128]
    float *sl = reinterpret_cast<float *>(xl + (size_t)held * nkb * 128);   // [held][nkb]
    if constexpr (MODE != F8_DENSE) {
        // quantise this expert's rows while the weights arrive
        const int g = threadIdx.x >> 4, c = threadIdx.x & 15;
        for (int i = g; i < rows * nkb; i += 16) {
            const int r = i / nkb, kb = i - r * nkb;
            if constexpr (MODE == F8_GATEUP) {
                const int t = a.perm[row0 + r] / a.k;
                quant_row_lds(static_cast<const f16 *>(a.src) + (int64_t)t * K, K, kb, c,
                              xl + (size_t)r * nkb * 128, sl + r * nkb);
            } else {
                quant_row_lds(static_cast<const float *>(a.src) + (int64_t)(row0 + r) * K, K, kb,
                              c, xl + (size_t)r * nkb * 128, sl + r * nkb);
            }
        }
        lds_barrier();
    }
    const int rl = min(col, rows - 1);   // decode: this lane's row
    const uint8_t *xr = xl + rl * nkb * 128;
    const float *xsr = sl + rl * nkb;
    const int sw = (col >> 1) & 7;   // f of every fragment's row col
    const int o0 = (q ^ sw) * 16, o1 = ((q + 4) ^ sw) * 16;
    const int rounds = (nkb + 3) / 4;
    for (int j = 0; j < rounds; ++j) {
        const int kb = block_of(j);
        const bool in = 4 * j + wave < nkb;
        wait_vm<0>();   // block j has landed
        const float *scl = reinterpret_cast<const float *>(st + (4 + XR) * 1024);
        float sc[2] = {scl[32], scl[33]}, xs[MT];
        sc[0] = in ? sc[0] : 0.0f;
        sc[1] = in ? sc[1] : 0.0f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
            xs[m] = MODE == F8_DENSE ? scl[m * 16 + col] : xsr[kb];
        half32 wh[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const uint8_t *r = st + (f * 16 + col) * 128;
            wh[f] = f8_to_f16(join16(*reinterpret_cast<const int4_t *>(r + o0),
                                     *reinterpret_cast<const int4_t *>(r + o1)));
        }
        const int c0 = kb * 128 + q * 16;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            int4_t x0, x1;
            if constexpr (MODE == F8_DENSE) {
                const uint8_t *r = st + 4096 + (m * 16 + col) * 128;
                x0 = *reinterpret_cast<const int4_t *>(r + o0);
                x1 = *reinterpret_cast<const int4_t *>(r + o1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {   // bytes past K count as zeros
                    x0[i] = c0 < K ? x0[i] : 0;
                    x1[i] = c0 + 64 < K ? x1[i] : 0;
                }
            } else {   // zero-filled to whole blocks
                x0 = *reinterpret_cast<const int4_t *>(xr + c0);
                x1 = *reinterpret_cast<const int4_t *>(xr + c0 + 64);
            }
            const half32 xf = f8_to_f16(join16(x0, x1));
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const float4_t t = mfma_f16(wh[f], xf);
                const float s = xs[m] * sc[f];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[f][m][i] = __builtin_fmaf(t[i], s, acc[f][m][i]);
            }
        }
        wave_lds_sync();   // the stage is read
        issue(j + 1);      // without a branch: past the end the last block again
    }
    wait_vm<0>();
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            *reinterpret_cast<float4_t *>(red[wave][f * MT + m][lane]) = acc[f][m];
    __syncthreads();
    // fragment (f, m) is summed and stored by wave (f * MT + m) % 4; gate and
    // up of a fragment meet in one wave
    auto total = [&](int i) {
        float4_t v = *reinterpret_cast<const float4_t *>(red[0][i][lane]);
#pragma unroll
        for (int w = 1; w < 4; ++w)
            v += *reinterpret_cast<const float4_t *>(red[w][i][lane]);
        return v;
    };
    if constexpr (MODE == F8_GATEUP) {
        if (wave == 0 && col < rows) {
            const float4_t g = total(0), u = total(1);
            float4_t h;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = swiglu_fast(g[i], u[i]);
            *reinterpret_cast<float4_t *>(static_cast<float *>(a.out) + (int64_t)(row0 + col) * a.N +
                                          n0 + q * 4) = h;
        }
    } else {
        for (int i = wave; i < 2 * MT; i += 4) {
            const int f = i / MT, m = i - f * MT;
            const int r = m * 16 + col, n = n0 + f * 16 + q * 4;
            const float4_t v = total(i);
            if (r < rows && n < a.N)
                store4(a.out, MODE == F8_DOWN ? MOE_DTYPE_F16 : a.odt,
                       (int64_t)(row0 + r) * a.ldo + n, v, a.N - n,
                       MODE == F8_DOWN || (a.ldo % 4 == 0 && ((uintptr_t)a.out & 15) == 0));
        }
    }
}

template <int MODE, int MT>
static int launch_rows(const Fp8Args &a, dim3 grid, size_t lds, hipStream_t s)
{
    lds += (size_t)4 * f8_rows_stage<MODE, MT>();
    static LdsLimit limit;
    const int rc = limit.raise((const void *)fp8_rows_kernel<MODE, MT>,
                               (160 - 8 * MT) * 1024);   // beside the waves' sums
    if (rc)
        return rc;
    static_assert(4 * f8_rows_stage<MODE, MT>() +
                      (MODE == F8_DENSE ? 0 : FP8_DECODE_BLOCKS * 132) <= (160 - 8 * MT) * 1024,
                  "LDS of one workgroup");
    hipLaunchKernelGGL((fp8_rows_kernel<MODE, MT>), grid, dim3(256), lds, s, a);
    MOE_LAUNCH_CHECK("fp8_rows_kernel");
    return MOE_OK;
}

// Dense, any M, in row tiles of 16 or 32 (64-row tiles: 333 x 1408 x 2000
// takes 12 us against 7).
int launch_fp8_rows_dense(const Fp8Args &a, hipStream_t s)
{
    const unsigned nt = (unsigned)((a.N + 31) / 32);
    if (a.M <= 16)
        return launch_rows<F8_DENSE, 1>(a, dim3(nt, 1), 0, s);
    return launch_rows<F8_DENSE, 2>(a, dim3(nt, (unsigned)((a.M + 31) / 32)), 0, s);
}

// Decode experts: gate/up with SwiGLU into fp32 h, then down.
int launch_fp8_decode(Fp8Args a, const void *x_f16, float *h, int H, int I, const int64_t off[6],
                      void *y, hipStream_t s)
{
    auto lds = [&](int K) {
        return (size_t)std::min(a.T, FP8_DECODE_ROWS) * ((K + 127) / 128) * (128 + 4);
    };
    a.src = x_f16;
    a.out = h;
    a.N = I;
    a.K = H;
    a.off_w0 = off[0];
    a.off_w1 = off[1];
    a.off_s0 = off[3];
    a.off_s1 = off[4];
    const unsigned n = (unsigned)(a.T * a.k);
    const int rc = launch_rows<F8_GATEUP, 1>(a, dim3((I + 15) / 16, n), lds(H), s);
    if (rc)
        return rc;
    a.src = h;
    a.out = y;
    a.N = H;
    a.K = I;
    a.ldo = H;
    a.off_w0 = a.off_w1 = off[2];
    a.off_s0 = a.off_s1 = off[5];
    return launch_rows<F8_DOWN, 1>(a, dim3((H + 31) / 32, n), lds(I), s);
}

}  // namespace moe
