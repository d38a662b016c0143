// k_fp8_frag.h -- device helpers of the block-scaled FP8 (e4m3) kernels.
//
// Matrix core: v_mfma_f32_16x16x128_f8f6f4, one instruction per 128-long
// block of K, so a block's products are summed inside one accumulation from
// zero and scaled once afterwards.  Lane l holds, of each operand, row l % 16
// and 32 of the 128 K bytes.  Which bytes does not matter as long as both
// operands agree; here lane group q = l / 16 takes bytes 16q..16q+15 and
// 64+16q..64+16q+15, so that one 16-byte load of a wave covers 64 consecutive
// bytes of each of 16 rows (and a K that ends at the middle of a block drops
// the second piece).  Result: column l % 16 (second operand's row), rows
// 4q..4q+3 (first operand's).  The weights are the first operand, so a lane
// holds four consecutive output columns of one token.
#pragma once

#include "moe_common.h"

namespace moe {

typedef int int8_8 __attribute__((ext_vector_type(8)));   // 32 e4m3 values
typedef int int4_t __attribute__((ext_vector_type(4)));
typedef int int2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float4_t mfma_f8(int8_8 a, int8_8 b)
{
    const float4_t z = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ int8_8 join16(int4_t lo, int4_t hi)
{
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 32 e4m3 values as fp16 (exact: fp16 has the wider exponent and mantissa).
struct half32 {
    half8_t v[4];
};
// Pair u (0..15) of them: one conversion.
__device__ __forceinline__ void f8_pair(half32 &r, int8_8 x, int u)
{
    const half2_t a = u & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[u >> 1], 1.0f, true)
                            : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[u >> 1], 1.0f, false);
    r.v[u >> 2][2 * (u & 3)] = a[0];
    r.v[u >> 2][2 * (u & 3) + 1] = a[1];
}
__device__ __forceinline__ half32 f8_to_f16(int8_8 x)
{
    half32 r;
#pragma unroll
    for (int u = 0; u < 16; ++u)
        f8_pair(r, x, u);
    return r;
}

// The block's sum on the fp16 matrix instruction: four steps of 32, fp32
// accumulation.
__device__ __forceinline__ float4_t mfma_f16(const half32 &a, const half32 &b)
{
    float4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[j], b.v[j], c, 0, 0, 0);
    return c;
}

// Scale of a block of largest magnitude amax: amax / 448 (e4m3's largest
// value), at least 2^-126 so that its reciprocal is finite; 0 for a block of
// zeros; with pow2 the next power of two (then x / s is exact and only e4m3
// rounding remains).
__device__ __forceinline__ float fp8_scale(float amax, bool pow2)
{
    float s = fmaxf(amax / 448.0f, 1.1754943508222875e-38f);
    if (pow2) {
        const uint32_t b = __builtin_bit_cast(uint32_t, s);
        s = __builtin_bit_cast(float, (b & 0x7fffffu) ? (b & 0x7f800000u) + 0x800000u : b);
    }
    return amax > 0.0f ? s : 0.0f;
}

// 1 / s of a power-of-two scale (exact); 0 for s = 0.
__device__ __forceinline__ float fp8_inv_pow2(float s)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, s);
    return b ? __builtin_bit_cast(float, 0x7f000000u - b) : 0.0f;
}

// Four values (already divided by the scale, |v| <= 448) to e4m3, nearest even.
__device__ __forceinline__ int fp8_pack4(float a, float b, float c, float d)
{
    int r = 0;
    r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    return r;
}

// Largest value over the 16 lanes of a row.
__device__ __forceinline__ float row16_max(float a)
{
#define MOE_ROW_MAX(C)                                                                        \
    a = fmaxf(a, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(                       \
                     0, __builtin_bit_cast(int, a), C, 0xF, 0xF, false)))
    MOE_ROW_MAX(0xB1);
    MOE_ROW_MAX(0x4E);
    MOE_ROW_MAX(0x141);
    MOE_ROW_MAX(0x140);
#undef MOE_ROW_MAX
    return a;
}

enum { F8_DENSE = 0, F8_GATEUP = 1, F8_DOWN = 2 };
constexpr int FP8_DECODE_MAX_T = 128;   // routed experts: decode kernels up to this many tokens,
constexpr int FP8_DECODE_ROWS = 16;     // of an expert in a workgroup,
constexpr int FP8_DECODE_BLOCKS = 600;  // whose quantised rows are as many 128-blocks (132 bytes) in LDS
// A launch has fewer than 2^32 threads: tiles of 512 threads (in whole groups of
// the 8 XCDs), 128-blocks of tokens of 16 threads (and one workgroup more).
constexpr int FP8_MOST_TILES = (1 << 23) - 8;
constexpr int FP8_MOST_TOKEN_BLOCKS = (1 << 28) - 32;

// One row tile of the routed experts: its expert's blob, first sorted row and
// rows.  Entry 0 of a table holds the number of tiles in `rows`.
struct Fp8TileRec {
    const uint8_t *blob;
    int32_t row0, rows;
};

struct Fp8Args {
    // tokens: e4m3 rows of ldx bytes and their scales, one per 128 columns
    const uint8_t *x;
    const float *xs;
    int64_t ldx;
    // dense weights
    const uint8_t *w;
    const float *ws;
    int64_t ldw;
    // routed experts: device table of blobs, section offsets inside a blob
    const void *const *blobs;
    int64_t off_w0, off_w1, off_s0, off_s1;
    const int32_t *offsets, *perm;
    const Fp8TileRec *tiles;
    const void *src;        // decode: fp16 tokens (gate/up) or fp32 h (down)
    int E, k, T;
    int M, N, K;            // rows, output columns (gate/up: I), contraction length
    void *out;
    int64_t ldo;
    float *hs;              // gate/up: scales of the quantised h
    int odt;                // dense: output dtype
};

// Stores four consecutive output columns of one row in the output's dtype.
__device__ __forceinline__ void store4(void *out, int dt, int64_t at, float4_t v, int n, bool vec)
{
    if (dt == MOE_DTYPE_F32) {
        float *p = static_cast<float *>(out) + at;
        if (vec && n >= 4) {
            *reinterpret_cast<float4_t *>(p) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n)
                    p[i] = v[i];
        }
        return;
    }
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = dt == MOE_DTYPE_F16 ? __builtin_bit_cast(uint16_t, (f16)v[i])
                                   : __builtin_bit_cast(uint16_t, (__bf16)v[i]);
    }
    uint16_t *p = static_cast<uint16_t *>(out) + at;
    if (vec && n >= 4) {
        int2_t u;
        u[0] = (int)(h[0] | ((uint32_t)h[1] << 16));
        u[1] = (int)(h[2] | ((uint32_t)h[3] << 16));
        *reinterpret_cast<int2_t *>(p) = u;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n)
                p[i] = h[i];
    }
}

}  // namespace moe
