// k_linear_rows.hip -- fp16 products of up to 16 rows (decode), out = residual +
// act(x w^T + bias): bound by the stream of the weights.
//
// A workgroup of eight waves forms 16 columns: each wave takes every eighth block of
// 64 k and loads weights and tokens straight into the matrix instruction's layout, so
// that everything it needs for four blocks is in flight at once and nothing waits at
// a barrier before the waves' sums meet in LDS.  (Lanes then read 16 bytes of 16
// different rows, which the L1 serves at a quarter of its rate: 34 GB/s a compute
// unit, still more than its share of memory.  Staged through LDS by tiles of 16 x 32,
// 8 groups of waves and three stages: 8.3 us for one row of 5632 x 2048 out of
// memory; so 6.5.)
#include <algorithm>

#include "k_linear.h"

namespace moe {

constexpr int LR_WAVES = 8, LR_UNROLL = 4;

// Two steps of 32 k: block b of the lane's row, zeros behind K.
struct LrPair {
    half8_t v[2];
};
__device__ __forceinline__ LrPair lr_load(const f16 *row, int b, int K)
{
    LrPair r;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int k = b * 64 + s * 32 + ((threadIdx.x & 63) >> 4) * 8;
        const half8_t v = ldg(reinterpret_cast<const half8_t *>(row + min(k, K - 8)));
        r.v[s] = k < K ? v : half8_t{};
    }
    return r;
}

template <typename T>
__global__ __launch_bounds__(64 * LR_WAVES) void linear_rows_kernel(LinArgs a)
{
    __shared__ float red[LR_WAVES][16][17];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, q = lane >> 4;
    const int nkb = (a.K + 63) / 64;
    const f16 *x = a.a + min(col, a.M - 1) * a.lda;
    for (int64_t n0 = (int64_t)blockIdx.x * 16; n0 < a.N; n0 += (int64_t)gridDim.x * 16) {
        const f16 *w = a.b + min(n0 + col, (int64_t)a.N - 1) * a.ldb;
        float4_t acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        int b = wave;
        for (; b + (LR_UNROLL - 1) * LR_WAVES < nkb; b += LR_UNROLL * LR_WAVES) {
            LrPair wv[LR_UNROLL], xv[LR_UNROLL];
#pragma unroll
            for (int u = 0; u < LR_UNROLL; ++u)
                wv[u] = lr_load(w, b + u * LR_WAVES, a.K);
#pragma unroll
            for (int u = 0; u < LR_UNROLL; ++u)
                xv[u] = lr_load(x, b + u * LR_WAVES, a.K);
#pragma unroll
            for (int u = 0; u < LR_UNROLL; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    acc[s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv[u].v[s], xv[u].v[s], acc[s],
                                                                    0, 0, 0);
        }
        for (; b < nkb; b += LR_WAVES) {
            const LrPair wv = lr_load(w, b, a.K), xv = lr_load(x, b, a.K);
#pragma unroll
            for (int s = 0; s < 2; ++s)
                acc[s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv.v[s], xv.v[s], acc[s], 0, 0, 0);
        }
        acc[0] += acc[1];
#pragma unroll
        for (int i = 0; i < 4; ++i)   // a lane holds four columns of row `col`
            red[wave][col][q * 4 + i] = acc[0][i];
        __syncthreads();
        const int m = threadIdx.x >> 4;
        const int64_t n = n0 + (threadIdx.x & 15);
        if (m < a.M && n < a.N) {   // the waves' sums in their order
            float v = red[0][m][threadIdx.x & 15];
#pragma unroll
            for (int i = 1; i < LR_WAVES; ++i)
                v += red[i][m][threadIdx.x & 15];
            if (a.bias)
                v += a.bias[n];
            if (a.z)
                a.z[m * a.ldz + n] = (f16)v;
            v = act_value(v, a.act);
            if (a.residual)
                v += (float)static_cast<const T *>(a.residual)[m * a.ldr + n];
            static_cast<T *>(a.out)[m * a.ldo + n] = (T)v;
        }
        __syncthreads();
    }
}

int launch_linear_rows(const LinArgs &a, hipStream_t s)
{
    const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)a.N + 15) / 16, 1 << 16);
    if (a.odt == MOE_DTYPE_F32)
        hipLaunchKernelGGL(linear_rows_kernel<float>, dim3(grid), dim3(64 * LR_WAVES), 0, s, a);
    else
        hipLaunchKernelGGL(linear_rows_kernel<f16>, dim3(grid), dim3(64 * LR_WAVES), 0, s, a);
    MOE_LAUNCH_CHECK("linear_rows_kernel");
    return MOE_OK;
}

}  // namespace moe
