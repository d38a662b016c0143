// k_linear_rows.hip -- fp16 products of one or two rows (decode), out = residual +
// act(x w^T + bias): bound by the stream of the weights.
//
// A wave takes a row of the weights and walks k with its 64 lanes side by side (1 KB
// of the row an instruction, four in flight), each lane multiplying its eight k with
// those of the tokens (v_dot2_f32_f16, fp32 sums); the lanes meet at the end.  No
// LDS, no barrier.  Out of memory, in a captured run of calls: one row of 5632 x 2048
// 5.9 us (3.9 TB/s), of 11264 x 2048 9.8 (4.7), two rows 6.5 and 10.6; for more rows
// the tokens' loads and sums outweigh the stream (four 8.9, eight 11, sixteen 17),
// and the 16-row tiles (8.4 to 9.2 for any of them, out of memory too) are faster.
#include <algorithm>
#include <type_traits>

#include "k_linear.h"

namespace moe {

template <typename T, int MT>
__global__ __launch_bounds__(256) void linear_rows_kernel(LinArgs a)
{
    constexpr int U = 4;   // chunks in flight
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // (a wave past the last row repeats it and stores nothing: without a branch here
    // the arguments arrive together)
    const int n = min((int)blockIdx.x * 4 + wave, a.N - 1);
    const f16 *w = a.b + n * a.ldb, *x[MT];
    float acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        x[m] = a.a + min(m, a.M - 1) * a.lda;
        acc[m] = 0.0f;
    }
    // U chunks of 512 k from k0 on; CUT: they may reach past K
    auto chunks = [&](int k0, auto cut) {
        constexpr bool CUT = decltype(cut)::value;
        half8_t wv[U];
        auto at = [&](int u) {
            const int k = k0 + u * 512 + lane * 8;
            return CUT ? min(k, a.K - 8) : k;
        };
#pragma unroll
        for (int u = 0; u < U; ++u)
            wv[u] = ldg(reinterpret_cast<const half8_t *>(w + at(u)));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = !CUT || k0 + u * 512 + lane * 8 < a.K;
            if (CUT)
                wv[u] = in ? wv[u] : half8_t{};
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                half8_t xv = ldg(reinterpret_cast<const half8_t *>(x[m] + at(u)));
                if (CUT)
                    xv = in ? xv : half8_t{};
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    acc[m] = dot2(half2_t{wv[u][j], wv[u][j + 1]}, half2_t{xv[j], xv[j + 1]},
                                  acc[m]);
            }
        }
    };
    const bool stores = lane < a.M && (int)blockIdx.x * 4 + wave < a.N;
    const float bias = a.bias ? a.bias[n] : 0.0f;
    const float res = a.residual && stores
                          ? (float)static_cast<const T *>(a.residual)[lane * a.ldr + n] : 0.0f;
    int k0 = 0;
    for (; k0 + U * 512 <= a.K; k0 += U * 512)
        chunks(k0, std::false_type());
    if (k0 < a.K)
        chunks(k0, std::true_type());
    float v = 0.0f;   // lane m: row m's
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const float s = wave_sum_f32(acc[m]);
        v = lane == m ? s : v;
    }
    if (stores) {
        v += bias;
        if (a.z)
            a.z[lane * a.ldz + n] = (f16)v;
        static_cast<T *>(a.out)[lane * a.ldo + n] = (T)(act_value(v, a.act) + res);
    }
}

template <typename T>
static void launch_rows_t(LinArgs a, hipStream_t s)
{
    // a launch has fewer than 2^32 threads: columns beyond that take another
    const int most = 1 << 25;
    for (int left = a.N; left > 0; left -= most) {
        a.N = std::min(left, most);
        const unsigned grid = (unsigned)((a.N + 3) / 4);
        if (a.M == 1)
            hipLaunchKernelGGL((linear_rows_kernel<T, 1>), dim3(grid), dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((linear_rows_kernel<T, 2>), dim3(grid), dim3(256), 0, s, a);
        a.b += most * a.ldb;
        a.bias = a.bias ? a.bias + most : nullptr;
        a.z = a.z ? a.z + most : nullptr;
        a.residual = a.residual ? static_cast<const T *>(a.residual) + most : nullptr;
        a.out = static_cast<T *>(a.out) + most;
    }
}

int launch_linear_rows(const LinArgs &a, hipStream_t s)
{
    if (a.odt == MOE_DTYPE_F32)
        launch_rows_t<float>(a, s);
    else
        launch_rows_t<f16>(a, s);
    MOE_LAUNCH_CHECK("linear_rows_kernel");
    return MOE_OK;
}

}  // namespace moe
