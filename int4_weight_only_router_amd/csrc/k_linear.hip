// k_linear.hip -- fp16 matrix products with bias, activation and residual in
// their epilogue, and their gradients:
//
//   z = x w^T + bias,  out = residual + act(z)
//   dz = dy act'(z),   dx = dz w,   dw = dz^T x,   dbias = sum_m dz
#include <algorithm>

#include "k_linear.h"

namespace moe {

__device__ __forceinline__ float out_value(const void *p, int dt, int64_t at)
{
    return dt == MOE_DTYPE_F32 ? static_cast<const float *>(p)[at]
                               : (float)static_cast<const f16 *>(p)[at];
}

__device__ __forceinline__ void epilogue1(const LinArgs &a, int m, int n, float v)
{
    if (m >= a.M || n >= a.N)
        return;
    if (a.bias)
        v += a.bias[n];
    if (a.z)
        a.z[m * a.ldz + n] = (f16)v;
    v = act_value(v, a.act);
    if (a.residual)
        v += out_value(a.residual, a.odt, m * a.ldr + n);
    if (a.odt == MOE_DTYPE_F32)
        static_cast<float *>(a.out)[m * a.ldo + n] = v;
    else
        static_cast<f16 *>(a.out)[m * a.ldo + n] = (f16)v;
}

// 64 x 64 tiles of four waves, K in steps of 32 through LDS.
__global__ __launch_bounds__(256) void linear_kernel(LinArgs a)
{
    __shared__ __align__(16) f16 as[64][40], bs[64][40];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
    float4_t acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        acc[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < a.K; k0 += 32) {
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * 32; i += 256) {
            const int ra = a.a_ks ? i & 63 : i >> 5, ka = a.a_ks ? i >> 6 : i & 31;
            const bool in_a = m0 + ra < a.M && k0 + ka < a.K;
            const int64_t at_a = a.a_ks ? (k0 + ka) * a.lda + m0 + ra : (m0 + ra) * a.lda + k0 + ka;
            as[ra][ka] = in_a ? a.a[at_a] : (f16)0.0f;
            const int rb = a.b_ks ? i & 63 : i >> 5, kb = a.b_ks ? i >> 6 : i & 31;
            const bool in_b = n0 + rb < a.N && k0 + kb < a.K;
            const int64_t at_b = a.b_ks ? (k0 + kb) * a.ldb + n0 + rb : (n0 + rb) * a.ldb + k0 + kb;
            bs[rb][kb] = in_b ? a.b[at_b] : (f16)0.0f;
        }
        __syncthreads();
        const int r = lane & 15, q = (lane >> 4) * 8;
        const half8_t x = *reinterpret_cast<const half8_t *>(&as[wave * 16 + r][q]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const half8_t w = *reinterpret_cast<const half8_t *>(&bs[i * 16 + r][q]);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x, acc[i], 0, 0, 0);
        }
    }
    // a lane holds four consecutive columns of one row
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            epilogue1(a, m0 + wave * 16 + (lane & 15), n0 + i * 16 + (lane >> 4) * 4 + j, acc[i][j]);
}

size_t linear_ws(int, int, int) { return 0; }

int launch_linear(const LinArgs &a, void *, hipStream_t s)
{
    hipLaunchKernelGGL(linear_kernel, dim3((a.N + 63) / 64, (a.M + 63) / 64), dim3(256), 0, s, a);
    MOE_LAUNCH_CHECK("linear_kernel");
    return MOE_OK;
}

// dz = dy act'(z) in fp16 (rows of ldd, zeros behind column N) and its column
// sums over 64 rows, from the unrounded values.
constexpr int DZ_ROWS = 64;
__global__ __launch_bounds__(256) void linear_dz_kernel(LinGrads g, f16 *dz, int64_t ldd,
                                                        float *parts)
{
    const int n = blockIdx.x * 256 + threadIdx.x;
    const int64_t m0 = (int64_t)blockIdx.y * DZ_ROWS, m1 = min(m0 + DZ_ROWS, (int64_t)g.M);
    if (n >= ldd)
        return;
    float s = 0.0f;
    for (int64_t m = m0; m < m1; ++m) {
        float v = n < g.N ? (float)g.dy[m * g.lddy + n] : 0.0f;
        if (g.act != MOE_ACT_NONE && n < g.N)
            v *= act_grad((float)g.z[m * g.ldz + n], g.act);
        dz[m * ldd + n] = (f16)v;
        s += v;
    }
    if (parts && n < g.N)
        parts[(int64_t)blockIdx.y * g.N + n] = s;
}

__global__ __launch_bounds__(1024) void linear_dbias_kernel(const float *parts, int G, int N,
                                                            float *out)
{
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = blockIdx.x * 64 + lane;
    float v = 0.0f;
    if (n < N)
        for (int g = wave; g < G; g += 16)
            v += parts[(int64_t)g * N + n];
    s[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && n < N) {
        for (int i = 1; i < 16; ++i)
            v += s[i][lane];
        out[n] = v;
    }
}

static int64_t dz_ld(int N) { return ((int64_t)N + 7) / 8 * 8; }

size_t linear_backward_ws(int M, int N, int)
{
    return (size_t)al256((int64_t)M * dz_ld(N) * 2) +
           (size_t)((M + DZ_ROWS - 1) / DZ_ROWS) * N * 4;
}

int launch_linear_backward(const LinGrads &g, void *ws, hipStream_t s)
{
    const int64_t ldd = dz_ld(g.N);
    f16 *dz = static_cast<f16 *>(ws);
    float *parts = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) +
                                             al256((int64_t)g.M * ldd * 2));
    const int G = (g.M + DZ_ROWS - 1) / DZ_ROWS;
    if (g.M > 0) {
        hipLaunchKernelGGL(linear_dz_kernel, dim3((unsigned)((ldd + 255) / 256), G), dim3(256), 0, s,
                           g, dz, ldd, g.dbias ? parts : nullptr);
        MOE_LAUNCH_CHECK("linear_dz_kernel");
    }
    if (g.dbias) {
        hipLaunchKernelGGL(linear_dbias_kernel, dim3((g.N + 63) / 64), dim3(1024), 0, s, parts, G,
                           g.N, g.dbias);
        MOE_LAUNCH_CHECK("linear_dbias_kernel");
    }
    LinArgs a{};
    a.act = MOE_ACT_NONE;
    a.odt = g.odt;
    a.a = dz;
    a.lda = ldd;
    if (g.dx && g.M > 0) {
        a.b = g.w;
        a.ldb = g.ldw;
        a.b_ks = true;
        a.M = g.M;
        a.N = g.K;
        a.K = g.N;
        a.out = g.dx;
        a.ldo = g.lddx;
        const int rc = launch_linear(a, nullptr, s);
        if (rc)
            return rc;
    }
    if (g.dw) {
        a.a_ks = a.b_ks = true;
        a.b = g.x;
        a.ldb = g.ldx;
        a.M = g.N;
        a.N = g.K;
        a.K = g.M;
        a.out = g.dw;
        a.ldo = g.lddw;
        return launch_linear(a, nullptr, s);
    }
    return MOE_OK;
}

}  // namespace moe
