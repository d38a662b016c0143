// k_linear.h -- arguments and epilogue of the fp16 matrix products.
#pragma once

#include "k_block.h"

namespace moe {

// Column sums of partial sums [groups][n]: 64 columns a workgroup of WAVES waves, every
// 16th group together and those in their order, whatever the waves.
struct LinColumns {
    const float *parts;
    int groups, n;
    float *out;   // or null: none
};
template <int WAVES>
__device__ __forceinline__ void column_sums(const LinColumns &c, int block, float (*s)[64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = block * 64 + lane;
    float v[16 / WAVES];
#pragma unroll
    for (int i = 0; i < 16 / WAVES; ++i)
        v[i] = 0.0f;
    if (n < c.n) {
#pragma unroll 4
        for (int g = 0; g < c.groups; g += 16)
#pragma unroll
            for (int i = 0; i < 16 / WAVES; ++i) {
                const int at = g + i * WAVES + wave;   // (no branch between the loads)
                const float p = c.parts[(int64_t)min(at, c.groups - 1) * c.n + n];
                v[i] += at < c.groups ? p : 0.0f;
            }
    }
#pragma unroll
    for (int i = 0; i < 16 / WAVES; ++i)
        s[i * WAVES + wave][lane] = v[i];
    __syncthreads();
    if (wave == 0 && n < c.n) {
        float t = s[0][lane];
#pragma unroll
        for (int i = 1; i < 16; ++i)
            t += s[i][lane];
        c.out[n] = t;
    }
}

// out[m][n] = residual + act(sum_k A(m, k) B(n, k) + bias[n]).  An operand's
// rows either run along k ("kc": A(m, k) = a[m lda + k]) or across it ("ks":
// A(m, k) = a[k lda + m]).
struct LinArgs {
    const f16 *a, *b;
    int64_t lda, ldb;
    bool a_ks, b_ks;
    // b_ks: every k of b twice, for the two fp16 of a's; a_ks: one after the other, else
    // all of them over again
    bool twice;
    int M, N, K;
    const float *bias;
    int act;
    const void *residual;
    int64_t ldr;
    void *out;
    int odt;
    int64_t ldo;
    f16 *z;
    int64_t ldz;
    // tiles: k dealt out over `splits` workgroups, kblocks blocks of 64 each, whose
    // results lie split_stride elements apart
    int splits, kblocks;
    int64_t split_stride;
    LinColumns columns;   // of the launch that joins the splits
};

// How a product is computed: the form of its tiles, and k in `splits` parts whose
// sums a second launch joins.
struct LinPlan {
    int form, splits;
    int64_t items;   // workgroups
};
constexpr int64_t LIN_MOST_ITEMS = (1 << 22) - 8;   // a launch has fewer than 2^32 threads
// Offsets inside a tile of up to 256 rows are 32 bits wide; dz's rows hold two values for
// each of its columns.
constexpr int LIN_MOST_LD = 1 << 22;
constexpr int LIN_MOST_TWICE = 1 << 29;             // rows whose every k is passed twice
// across: operands whose rows run across k (b, then a too)
LinPlan linear_plan(int M, int N, int K, int across);
int launch_linear_tile(LinArgs, const LinPlan &, void *ws, hipStream_t);
constexpr int LIN_FEW_ROWS = 2;
int launch_linear_rows(const LinArgs &, hipStream_t);   // so many rows, both operands along k

// 1 / (1 + exp(-x)) by the hardware's exp2 and reciprocal (an ulp each).
__device__ __forceinline__ float logistic(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
}

// The normal distribution's function Phi(z), and e = exp(-z^2 / 2) on the way:
// Phi(-|z|) = e t P(t) with t = 1 / (1 + 0.32 |z|), P fitted here by weighted least
// squares to within 3.2e-8 of it over all z; in fp32 z Phi(z) is off by less than four
// half steps of |z|.  One exp2 and one reciprocal, for the gradient too; the library's
// erff takes both of its branches wherever a wave's lanes differ.
__device__ __forceinline__ float normal_cdf(float z, float &e)
{
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.32f, fabsf(z), 1.0f));
    float p = -0.021078196f;
    p = __builtin_fmaf(p, t, 0.095407377f);
    p = __builtin_fmaf(p, t, -0.146707672f);
    p = __builtin_fmaf(p, t, 0.065328231f);
    p = __builtin_fmaf(p, t, -0.009377686f);
    p = __builtin_fmaf(p, t, 0.058654003f);
    p = __builtin_fmaf(p, t, 0.087829092f);
    p = __builtin_fmaf(p, t, 0.114622360f);
    p = __builtin_fmaf(p, t, 0.127660946f);
    p = __builtin_fmaf(p, t, 0.127661529f);
    e = __builtin_amdgcn_exp2f(-0.72134752044f * (z * z));
    const float tail = p * t * e;
    return z < 0.0f ? tail : 1.0f - tail;
}

// Activations and their derivatives in fp32.  The tanh form of GELU by (1 + tanh u) / 2
// = logistic(2 u), with 2 u = GELU_A z (1 + GELU_B z^2).
constexpr float GELU_A = 1.5957691216057308f, GELU_B = 0.044715f;

__device__ __forceinline__ float act_value(float z, int act)
{
    switch (act) {
    case MOE_ACT_RELU:
        return z < 0.0f ? 0.0f : z;   // (NaN stays)
    case MOE_ACT_SILU:
        return z * logistic(z);
    case MOE_ACT_GELU: {
        float e;
        return z * normal_cdf(z, e);
    }
    case MOE_ACT_GELU_TANH:
        return z * logistic(GELU_A * __builtin_fmaf(GELU_B * z * z, z, z));
    default:
        return z;
    }
}

// (z comes as fp16: one that left its range is an infinity, where the products of zero
// and z below would be NaN; the derivatives there are those of fp16's last value)
__device__ __forceinline__ float act_grad(float z, int act)
{
    z = fabsf(z) > 65504.0f ? copysignf(65504.0f, z) : z;   // (NaN stays)
    switch (act) {
    case MOE_ACT_RELU:
        return z > 0.0f ? 1.0f : 0.0f;
    case MOE_ACT_SILU: {
        const float s = logistic(z);
        return s * (1.0f + z * (1.0f - s));
    }
    case MOE_ACT_GELU: {
        float e;
        const float c = normal_cdf(z, e);
        return __builtin_fmaf(z * 0.39894228040143268f, e, c);
    }
    case MOE_ACT_GELU_TANH: {
        const float s = logistic(GELU_A * __builtin_fmaf(GELU_B * z * z, z, z));
        return s * (1.0f + z * (1.0f - s) * GELU_A * __builtin_fmaf(3.0f * GELU_B * z, z, 1.0f));
    }
    default:
        return 1.0f;
    }
}

// One call's plan (items of LIN_MOST_ITEMS + 1 and more: no launch holds them).
LinPlan linear_forward_plan(int M, int N, int K);
size_t linear_ws(const LinPlan &, int M, int N);
int launch_linear(const LinArgs &, const LinPlan &, void *ws, hipStream_t);
struct LinGradPlan {
    LinPlan dx, dw;
    bool fits;
    bool fits2;   // the products with dz as the sum of two fp16
    LinPlan dx2, dw2;
    int64_t col, parts, products, total;   // workspace (dz, or its form for dx, stands first)
};
LinGradPlan linear_grad_plan(int M, int N, int K);
// Whether an activation leaves dz an fp16 as it is.
inline bool linear_dz_exact(int act) { return act == MOE_ACT_NONE || act == MOE_ACT_RELU; }
struct LinGrads {
    const f16 *dy, *z, *x, *w;
    int64_t lddy, ldz, ldx, ldw;
    int act, M, N, K;
    void *dx, *dw;
    int64_t lddx, lddw;
    int odt;
    bool two;   // dz as the sum of two fp16
    float *dbias;
};
int launch_linear_backward(const LinGrads &, const LinGradPlan &, void *ws, hipStream_t);

}  // namespace moe
