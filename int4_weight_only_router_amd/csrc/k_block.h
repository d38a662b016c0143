// k_block.h -- what the kernels around a routed block share: loads and stores of
// columns in any activation type, rows as buffers, and the norms' arguments.
#pragma once

#include "moe_common.h"

namespace moe {

typedef __bf16 bf16;
typedef __bf16 bf168_t __attribute__((ext_vector_type(8)));

template <typename T>
struct Vec8;
template <>
struct Vec8<f16> { typedef half8_t type; };
template <>
struct Vec8<bf16> { typedef bf168_t type; };

// C values in a row, up to 16 bytes an instruction.
template <typename T, int C>
struct alignas(C * sizeof(T) < 16 ? C * sizeof(T) : 16) Piece {
    T v[C];
};

// Columns c .. c + C - 1 of a row; zeros from column `cols` on.  vec: rows are
// 16-byte aligned.
template <typename T, int C>
__device__ __forceinline__ void load_piece(const T *row, int c, int cols, bool vec, float (&v)[C])
{
    if (vec && c + C <= cols) {
        const Piece<T, C> a = *reinterpret_cast<const Piece<T, C> *>(row + c);
#pragma unroll
        for (int i = 0; i < C; ++i)
            v[i] = (float)a.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            v[i] = c + i < cols ? (float)row[c + i] : 0.0f;
    }
}

// The same columns, rounded once; those from `cols` on are left as they were.
template <typename T, int C>
__device__ __forceinline__ void store_piece(T *row, int c, int cols, bool vec, const float (&v)[C])
{
    if (vec && c + C <= cols) {
        Piece<T, C> a;
#pragma unroll
        for (int i = 0; i < C; ++i)
            a.v[i] = (T)v[i];
        *reinterpret_cast<Piece<T, C> *>(row + c) = a;
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (c + i < cols)
                row[c + i] = (T)v[i];
    }
}

// A row of `cols` values for buffer instructions, whose range check does without a
// branch, and without a lane mask, for every value: zeros are read past the row's end,
// and nothing is written there.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const T *row, int cols)
{
    constexpr int RAW = 0x00020000;   // 32-bit data, no swizzle
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(row), 0, cols * (int)sizeof(T), RAW);
}

// Rows of T x H.  vec: H a multiple of 8 and every tensor's rows 16-byte aligned.
struct NormArgs {
    const void *y, *residual, *gate, *post_w, *post_b, *pre_w, *pre_b;
    void *out, *n;
    int64_t ldy, ldr, ldg, ldo, ldn;   // ldg 0: one gate row for all
    float scale, eps;
    int T, H;
    bool layer, post, offset, w32, vec;
};

// Gradients, laid out as what they are gradients of; `sums`: fp32 [H] over the
// tokens (a shared gate's, the post norm's weight and bias, the pre norm's).
struct NormGrads {
    const void *dout, *dn;
    void *dy, *dresidual, *dgate;
    float *sums[5];
    float *parts;
    int nsums;
};

struct NormSums {
    float *p[5];
    int n;
};

int launch_block_norm(const NormArgs &, int dtype, hipStream_t);
size_t block_norm_backward_ws(int T, int H);
int launch_block_norm_backward(const NormArgs &, NormGrads, int dtype, hipStream_t);

}  // namespace moe
