// k_linear.h -- arguments and epilogue of the fp16 matrix products.
#pragma once

#include "k_block.h"

namespace moe {

// out[m][n] = residual + act(sum_k A(m, k) B(n, k) + bias[n]).  An operand's
// rows either run along k ("kc": A(m, k) = a[m lda + k]) or across it ("ks":
// A(m, k) = a[k lda + m]).
struct LinArgs {
    const f16 *a, *b;
    int64_t lda, ldb;
    bool a_ks, b_ks;
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
};

// Activations and their derivatives in fp32.
__device__ __forceinline__ float act_value(float z, int act)
{
    switch (act) {
    case MOE_ACT_RELU:
        return z > 0.0f ? z : z != z ? z : 0.0f;
    case MOE_ACT_SILU:
        return z / (1.0f + expf(-z));
    case MOE_ACT_GELU:
        return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case MOE_ACT_GELU_TANH:
        return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
    default:
        return z;
    }
}

__device__ __forceinline__ float act_grad(float z, int act)
{
    switch (act) {
    case MOE_ACT_RELU:
        return z > 0.0f ? 1.0f : 0.0f;
    case MOE_ACT_SILU: {
        const float s = 1.0f / (1.0f + expf(-z));
        return s * (1.0f + z * (1.0f - s));
    }
    case MOE_ACT_GELU:
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
               z * 0.39894228040143268f * expf(-0.5f * z * z);
    case MOE_ACT_GELU_TANH: {
        const float t = tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z));
        return 0.5f * (1.0f + t) +
               0.5f * z * (1.0f - t * t) * 0.79788456080286536f * (1.0f + 0.134145f * z * z);
    }
    default:
        return 1.0f;
    }
}

size_t linear_ws(int M, int N, int K);
size_t linear_backward_ws(int M, int N, int K);
int launch_linear(const LinArgs &, void *ws, hipStream_t);
struct LinGrads {
    const f16 *dy, *z, *x, *w;
    int64_t lddy, ldz, ldx, ldw;
    int act, M, N, K;
    void *dx, *dw;
    int64_t lddx, lddw;
    int odt;
    float *dbias;
};
int launch_linear_backward(const LinGrads &, void *ws, hipStream_t);

}  // namespace moe
