// k_block_norm.hip -- the end of one block and the start of the next:
//
//   u = post(y) or y,   r = residual + scale * gate * u,   n = pre(r)
//
// with RMS or layer norms, and its gradients.  One pass: a row stays in fp32
// registers from its loads to its stores, so every value is read once and
// written once, and n is formed from the unrounded r.  A layer norm's variance
// is the mean square of the centred values (a second sum over registers), not a
// difference of two large means.  Bound by memory.
#include <algorithm>

#include "k_block.h"

namespace moe {

// Sum over the row's threads: its wave, or all four waves of the workgroup.
// `part` alternates between two halves, so one barrier per sum suffices: a half
// is written again only behind the barrier of the sum in between.
template <int W>
__device__ __forceinline__ float row_sum(float v, float *part, int &half)
{
    v = wave_sum_f32(v);
    if constexpr (W == 1) {
        return v;
    } else {
        float *p = part + half * W;
        half ^= 1;
        if ((threadIdx.x & 63) == 0)
            p[threadIdx.x >> 6] = v;
        __syncthreads();
        return (p[0] + p[1]) + (p[2] + p[3]);
    }
}

// v normalised in place (columns past H hold zeros and stay so).
template <int W, int NC>
__device__ __forceinline__ void normalise(float (&v)[NC][8], int c0, const NormArgs &a, float *part,
                                          int &half)
{
    constexpr int STEP = W * 512;
    if (a.layer) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += v[i][j];
        const float mean = row_sum<W>(s, part, half) / (float)a.H;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = c0 + i * STEP + j < a.H ? v[i][j] - mean : 0.0f;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s = __builtin_fmaf(v[i][j], v[i][j], s);
    const float rho = 1.0f / sqrtf(row_sum<W>(s, part, half) / (float)a.H + a.eps);
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[i][j] *= rho;
}

// v * weight + bias; either may be absent.
template <typename WT, int NC, int STEP>
__device__ __forceinline__ void affine(float (&v)[NC][8], int c0, const NormArgs &a, const void *w,
                                       const void *b)
{
    const float one = a.offset ? 1.0f : 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = c0 + i * STEP;
        if (w) {
            float t[8];
            load8<WT>(static_cast<const WT *>(w), c, a.H, a.vec_w, t);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] *= t[j] + one;
        }
        if (b) {
            float t[8];
            load8<WT>(static_cast<const WT *>(b), c, a.H, a.vec_w, t);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] += t[j];
        }
    }
}

// W waves a row of up to 512 W NC columns: a wave a row (no barrier, all its
// loads in flight together) up to 2048 columns, above that the workgroup.
template <typename XT, typename WT, int W, int NC>
__global__ __launch_bounds__(256) void block_norm_kernel(NormArgs a)
{
    __shared__ float part[2 * W];
    constexpr int ROWS = 4 / W, STEP = W * 512;
    const int c0 = (W == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x) * 8;
    int half = 0;
    for (int64_t t = (int64_t)blockIdx.x * ROWS + (W == 1 ? threadIdx.x >> 6 : 0); t < a.T;
         t += (int64_t)gridDim.x * ROWS) {
        float r[NC][8], u[NC][8];
        if (a.residual) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                load8<XT>(static_cast<const XT *>(a.residual) + t * a.ldr, c0 + i * STEP, a.H,
                          a.vec_r, r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    r[i][j] = 0.0f;
        }
        if (a.y) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                load8<XT>(static_cast<const XT *>(a.y) + t * a.ldy, c0 + i * STEP, a.H, a.vec_y,
                          u[i]);
            if (a.post) {
                normalise<W, NC>(u, c0, a, part, half);
                affine<WT, NC, STEP>(u, c0, a, a.post_w, a.post_b);
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float g[8];
                if (a.gate)
                    load8<XT>(static_cast<const XT *>(a.gate) + t * a.ldg, c0 + i * STEP, a.H,
                              a.vec_g, g);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    r[i][j] = __builtin_fmaf(a.scale, a.gate ? g[j] * u[i][j] : u[i][j], r[i][j]);
            }
        }
        if (a.out) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                store8<XT>(static_cast<XT *>(a.out) + t * a.ldo, c0 + i * STEP, a.H, a.vec_o, r[i]);
        }
        if (a.n) {
            normalise<W, NC>(r, c0, a, part, half);
            affine<WT, NC, STEP>(r, c0, a, a.pre_w, a.pre_b);
#pragma unroll
            for (int i = 0; i < NC; ++i)
                store8<XT>(static_cast<XT *>(a.n) + t * a.ldn, c0 + i * STEP, a.H, a.vec_n, r[i]);
        }
    }
}

template <typename XT, typename WT>
static int launch_norm_t(const NormArgs &a, hipStream_t s)
{
    const int64_t rows = a.H <= 2048 ? 4 : 1;   // of a workgroup
    const int64_t grid = std::min<int64_t>((a.T + rows - 1) / rows, 1 << 20);   // the rest in its loop
#define MOE_N(W, NC)                                                                            \
    hipLaunchKernelGGL((block_norm_kernel<XT, WT, W, NC>), dim3((unsigned)grid), dim3(256), 0, s, a)
    if (a.H <= 512) MOE_N(1, 1);
    else if (a.H <= 1024) MOE_N(1, 2);
    else if (a.H <= 2048) MOE_N(1, 4);
    else if (a.H <= 4096) MOE_N(4, 2);
    else MOE_N(4, 4);
#undef MOE_N
    MOE_LAUNCH_CHECK("block_norm_kernel");
    return MOE_OK;
}

template <typename XT>
static int launch_norm_x(const NormArgs &a, bool w32, hipStream_t s)
{
    return w32 ? launch_norm_t<XT, float>(a, s) : launch_norm_t<XT, XT>(a, s);
}

int launch_block_norm(const NormArgs &a, int dtype, int w_dtype, hipStream_t s)
{
    const bool w32 = w_dtype == MOE_DTYPE_F32;
    if (dtype == MOE_DTYPE_F32)
        return launch_norm_t<float, float>(a, s);
    return dtype == MOE_DTYPE_F16 ? launch_norm_x<f16>(a, w32, s)
                                  : launch_norm_x<bf16>(a, w32, s);
}

// ------------------------------------------------------------------ gradients
//
// With x = a normed row, m its normalised values, rho the reciprocal root, w
// the weight and g = dn * w:
//   dx = rho (g - m mean(g m) [- mean(g) for a layer norm]),
//   dw = sum_t dn m,  db = sum_t dn.
// Eight columns a thread, W waves a row, so that a thread keeps its columns from
// row to row and the five sums over the tokens stay in its registers; the row
// groups of a workgroup meet in LDS at the end, the workgroups' sums in a second
// launch, both in a fixed order.

constexpr int NB_THREADS = 1024;
enum { NB_GATE = 0, NB_POST_W, NB_POST_B, NB_PRE_W, NB_PRE_B, NB_SUMS };

// Sums of two values over a row's W waves (groups of W waves in a row).
__device__ __forceinline__ void group_sum2(float &a, float &b, int W, float2 *part, int &half)
{
    a = wave_sum_f32(a);
    b = wave_sum_f32(b);
    if (W == 1)
        return;
    const int wave = threadIdx.x >> 6;
    float2 *p = part + half * (NB_THREADS / 64);
    half ^= 1;
    if ((threadIdx.x & 63) == 0)
        p[wave] = float2{a, b};
    __syncthreads();
    const int w0 = wave & ~(W - 1);
    float sa = 0.0f, sb = 0.0f;
    for (int i = 0; i < W; ++i) {
        const float2 v = p[w0 + i];
        sa += v.x;
        sb += v.y;
    }
    a = sa;
    b = sb;
}

// v to its normalised values; returns the reciprocal root (0 for a turn past the
// last row, whose zeros must stay zeros also where eps is 0).
__device__ __forceinline__ float normalise_group(float (&v)[8], int c, bool live, const NormArgs &a,
                                                 int W, float2 *part, int &half)
{
    float s = 0.0f, q = 0.0f;
    if (a.layer) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s += v[j];
        group_sum2(s, q, W, part, half);
        const float mean = s / (float)a.H;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = c + j < a.H ? v[j] - mean : 0.0f;
    }
    s = q = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        s = __builtin_fmaf(v[j], v[j], s);
    group_sum2(s, q, W, part, half);
    const float rho = live ? 1.0f / sqrtf(s / (float)a.H + a.eps) : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] *= rho;
    return rho;
}

// g = dn * w to the gradient of the normed row; m its normalised values.
__device__ __forceinline__ void norm_input_grad(float (&g)[8], const float (&m)[8], float rho,
                                                const NormArgs &a, int W, float2 *part, int &half)
{
    float s = 0.0f, q = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        s += g[j];
        q = __builtin_fmaf(g[j], m[j], q);
    }
    group_sum2(s, q, W, part, half);
    const float mean = a.layer ? s / (float)a.H : 0.0f, along = q / (float)a.H;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        g[j] = rho * (g[j] - mean - m[j] * along);
}

template <typename XT, typename WT>
__global__ __launch_bounds__(NB_THREADS) void block_norm_backward_kernel(NormArgs a, NormGrads d,
                                                                         int W)
{
    __shared__ float2 part[2 * (NB_THREADS / 64)];
    __shared__ float cols[NB_THREADS * 8];
    const int wave = threadIdx.x >> 6;
    const int groups = NB_THREADS / 64 / W;   // rows at a time
    const int grp = wave / W;
    const int c = ((wave - grp * W) * 64 + (threadIdx.x & 63)) * 8;
    const int H = a.H;
    const float one = a.offset ? 1.0f : 0.0f;
    int half = 0;
    float sum[NB_SUMS][8];
#pragma unroll
    for (int k = 0; k < NB_SUMS; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum[k][j] = 0.0f;
    // every group takes as many turns (its sums meet at barriers); one past the
    // last row works on zeros and stores nothing
    for (int64_t t0 = (int64_t)blockIdx.x * groups; t0 < a.T; t0 += (int64_t)gridDim.x * groups) {
        const int64_t t = t0 + grp;
        const int cols_in = t < a.T ? H : 0;   // columns that this thread may touch
        const int64_t row = t < a.T ? t : 0;
        float u[8], r[8], gate[8], pm[8], dr[8], g[8];
        float post_rho = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            u[j] = r[j] = pm[j] = dr[j] = 0.0f;
        if (a.residual)
            load8<XT>(static_cast<const XT *>(a.residual) + row * a.ldr, c, cols_in, a.vec_r, r);
        if (d.dout)
            load8<XT>(static_cast<const XT *>(d.dout) + row * a.ldo, c, cols_in, a.vec_o, dr);
        if (d.dn)
            load8<XT>(static_cast<const XT *>(d.dn) + row * a.ldn, c, cols_in, a.vec_n, g);
        if (a.y) {
            load8<XT>(static_cast<const XT *>(a.y) + row * a.ldy, c, cols_in, a.vec_y, u);
            if (a.gate)
                load8<XT>(static_cast<const XT *>(a.gate) + row * a.ldg, c, cols_in, a.vec_g, gate);
            if (a.post) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    pm[j] = u[j];
                post_rho = normalise_group(pm, c, t < a.T, a, W, part, half);
                float w[8], b[8];
                if (a.post_w)
                    load8<WT>(static_cast<const WT *>(a.post_w), c, H, a.vec_w, w);
                if (a.post_b)
                    load8<WT>(static_cast<const WT *>(a.post_b), c, H, a.vec_w, b);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    u[j] = a.post_w ? pm[j] * (w[j] + one) : pm[j];
                    u[j] = a.post_b && c + j < cols_in ? u[j] + b[j] : u[j];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                r[j] = __builtin_fmaf(a.scale, a.gate ? gate[j] * u[j] : u[j], r[j]);
        }
        if (d.dn) {
            const float rho = normalise_group(r, c, t < a.T, a, W, part, half);   // r: normalised from here
            float w[8];
            if (a.pre_w)
                load8<WT>(static_cast<const WT *>(a.pre_w), c, H, a.vec_w, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum[NB_PRE_W][j] = __builtin_fmaf(g[j], r[j], sum[NB_PRE_W][j]);
                sum[NB_PRE_B][j] += g[j];
                g[j] = a.pre_w ? g[j] * (w[j] + one) : g[j];
            }
            norm_input_grad(g, r, rho, a, W, part, half);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                dr[j] += g[j];
        }
        if (d.dresidual)
            store8<XT>(static_cast<XT *>(d.dresidual) + row * a.ldr, c, cols_in, a.vec_dr, dr);
        if (a.y) {
            float dg[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dr[j] = c + j < cols_in ? a.scale * dr[j] : 0.0f;   // of gate * u
                dg[j] = dr[j] * u[j];
                sum[NB_GATE][j] += dg[j];
                dr[j] = a.gate ? dr[j] * gate[j] : dr[j];   // of u
            }
            if (d.dgate && a.ldg)
                store8<XT>(static_cast<XT *>(d.dgate) + row * a.ldg, c, cols_in, a.vec_dg, dg);
            if (a.post) {
                float w[8];
                if (a.post_w)
                    load8<WT>(static_cast<const WT *>(a.post_w), c, H, a.vec_w, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sum[NB_POST_W][j] = __builtin_fmaf(dr[j], pm[j], sum[NB_POST_W][j]);
                    sum[NB_POST_B][j] += dr[j];
                    dr[j] = a.post_w ? dr[j] * (w[j] + one) : dr[j];
                }
                norm_input_grad(dr, pm, post_rho, a, W, part, half);
            }
            if (d.dy)
                store8<XT>(static_cast<XT *>(d.dy) + row * a.ldy, c, cols_in, a.vec_dy, dr);
        }
    }
    // the groups' sums, in the order of the groups
    float *to = d.parts + (int64_t)blockIdx.x * d.nsums * H;
#pragma unroll
    for (int k = 0; k < NB_SUMS; ++k) {
        if (!d.sums[k])
            continue;
        if (groups > 1) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                cols[j * NB_THREADS + threadIdx.x] = sum[k][j];
            __syncthreads();
            if (grp == 0)
                for (int i = 1; i < groups; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sum[k][j] += cols[j * NB_THREADS + i * W * 64 + threadIdx.x];
        }
        if (grp == 0)
            store8<float>(to, c, H, H % 4 == 0, sum[k]);
        to += H;
    }
}

// Column sums over the workgroups' partial sums [G][n][H]: 16 workgroups' rows
// at a time per column, joined in a fixed order.
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float *__restrict__ parts, int G,
                                                         int H, NormSums to)
{
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = blockIdx.x * 64 + lane;
    const int64_t n = to.n;
    float v = 0.0f;
    if (col < H)
        for (int g = wave; g < G; g += 16)
            v += parts[(g * n + blockIdx.y) * H + col];
    s[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && col < H) {
        for (int i = 1; i < 16; ++i)
            v += s[i][lane];
        to.p[blockIdx.y][col] = v;
    }
}

// Waves a row: the fewest (a power of two) that hold H columns, eight a lane.
static int norm_waves(int H)
{
    int w = 1;
    while (w * 512 < H)
        w *= 2;
    return w;
}

static int norm_backward_grid(int T, int H)
{
    const int rows = NB_THREADS / 64 / norm_waves(H);
    return (int)std::min<int64_t>(((int64_t)T + rows - 1) / rows, 256);
}

size_t block_norm_backward_ws(int T, int H)
{
    return (size_t)norm_backward_grid(T, H) * NB_SUMS * H * sizeof(float);
}

int launch_block_norm_backward(const NormArgs &a, NormGrads d, int dtype, int w_dtype,
                               hipStream_t s)
{
    const int W = norm_waves(a.H), G = norm_backward_grid(a.T, a.H);
    NormSums to{};
    for (int k = 0; k < NB_SUMS; ++k)
        if (d.sums[k])
            to.p[to.n++] = d.sums[k];
    d.nsums = to.n;
    if (a.T > 0) {
#define MOE_NB(XT, WT)                                                                           \
    hipLaunchKernelGGL((block_norm_backward_kernel<XT, WT>), dim3((unsigned)G), dim3(NB_THREADS), 0, \
                       s, a, d, W)
        const bool w32 = w_dtype == MOE_DTYPE_F32;
        if (dtype == MOE_DTYPE_F32) MOE_NB(float, float);
        else if (dtype == MOE_DTYPE_F16 && w32) MOE_NB(f16, float);
        else if (dtype == MOE_DTYPE_F16) MOE_NB(f16, f16);
        else if (w32) MOE_NB(bf16, float);
        else MOE_NB(bf16, bf16);
#undef MOE_NB
        MOE_LAUNCH_CHECK("block_norm_backward_kernel");
    }
    if (to.n) {   // without tokens: zeros
        hipLaunchKernelGGL(norm_sums_kernel, dim3((a.H + 63) / 64, to.n), dim3(1024), 0, s,
                           d.parts, G, a.H, to);
        MOE_LAUNCH_CHECK("norm_sums_kernel");
    }
    return MOE_OK;
}

}  // namespace moe
