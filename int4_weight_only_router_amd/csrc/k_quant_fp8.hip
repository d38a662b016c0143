// k_quant_fp8.hip -- quantisation to e4m3 with one fp32 scale per block.
//
//   a = max |x| of the block,  s = a / 448 (or the next power of two),
//   q = e4m3(x / s), nearest even;  x is about q * s.
//
// Blocks of 1 x 128 (activations) or 128 x 128 (weights).  One pass: a block
// is held in registers between its maximum and its codes.  Bound by memory:
// every value is read once and written once at one byte.  Rows: 16 lanes a
// block, so that a wave reads 512 values in a row and no value crosses LDS;
// 16384 x 1408 fp16 13.0 us (70 MB, 5.4 TB/s; a large copy reaches 5.15).
// Weight blocks: a workgroup a block, 64 values a thread; 5632 x 2048 fp32
// 13.9 us (58 MB, 4.1 TB/s).
#include <algorithm>

#include "k_fp8_frag.h"

namespace moe {

template <typename XT>
__device__ __forceinline__ float to_f32(XT v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<f16>(f16 v) { return (float)v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v)   // bf16 bits
{
    return __builtin_bit_cast(float, (uint32_t)v << 16);
}

// Eight consecutive values from column c of a row; zeros past `cols`.
template <typename XT, bool VEC>
__device__ __forceinline__ void load8(const XT *row, int c, int cols, float (&v)[8])
{
    if (VEC && c + 8 <= cols) {
        if constexpr (sizeof(XT) == 4) {
            const float4_t a = *reinterpret_cast<const float4_t *>(row + c);
            const float4_t b = *reinterpret_cast<const float4_t *>(row + c + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        } else {
            typedef XT xt8 __attribute__((ext_vector_type(8)));
            const xt8 a = *reinterpret_cast<const xt8 *>(row + c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = to_f32<XT>(a[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = c + i < cols ? to_f32<XT>(row[c + i]) : 0.0f;
    }
}

// Divides by the scale and stores eight codes.
__device__ __forceinline__ void store8(uint8_t *row, int c, int cols, const float (&v)[8], float s,
                                       bool pow2, bool vec)
{
    float d[8];
    if (pow2 && s < __builtin_inff()) {
        const float inv = fp8_inv_pow2(s);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            d[i] = v[i] * inv;
    } else {
        const float z = s > 0.0f ? s : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            d[i] = v[i] / z;
    }
    int2_t q;
    q[0] = fp8_pack4(d[0], d[1], d[2], d[3]);
    q[1] = fp8_pack4(d[4], d[5], d[6], d[7]);
    if (vec && c + 8 <= cols) {
        *reinterpret_cast<int2_t *>(row + c) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols)
                row[c + i] = (uint8_t)((uint32_t)q[i >> 2] >> (8 * (i & 3)));
    }
}

__device__ __forceinline__ float max8(const float (&v)[8])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = fmaxf(m, fabsf(v[i]));
    return m;
}

// 1 x 128 blocks: 16 lanes per block, eight values each.
template <typename XT, bool VEC>
__global__ __launch_bounds__(256) void quant_rows_kernel(const XT *__restrict__ x, int64_t ldx,
                                                         int64_t rows, int cols, bool pow2,
                                                         uint8_t *__restrict__ q, int64_t ldq,
                                                         float *__restrict__ scales, bool vecq)
{
    const int nb = (cols + 127) / 128;
    const int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4;
    if (b >= rows * nb)
        return;   // whole 16-lane rows leave together
    const int64_t r = b / nb;
    const int kb = (int)(b - r * nb);
    const int c = kb * 128 + (threadIdx.x & 15) * 8;
    float v[8];
    load8<XT, VEC>(x + r * ldx, c, cols, v);
    const float s = fp8_scale(row16_max(max8(v)), pow2);
    if ((threadIdx.x & 15) == 0)
        scales[b] = s;
    store8(q + r * ldq, c, cols, v, s, pow2, vecq);
}

// 128 x 128 blocks: one workgroup per block, 8 rows of 8 values per thread.
template <typename XT, bool VEC>
__global__ __launch_bounds__(256) void quant_blocks_kernel(const XT *__restrict__ x, int64_t ldx,
                                                           int64_t rows, int cols, bool pow2,
                                                           uint8_t *__restrict__ q, int64_t ldq,
                                                           float *__restrict__ scales, bool vecq)
{
    __shared__ float top[4];
    const int nb = (cols + 127) / 128;
    const int64_t rb = blockIdx.x / nb;
    const int kb = (int)(blockIdx.x - rb * nb);
    const int c = kb * 128 + (threadIdx.x & 15) * 8;
    const int64_t r0 = rb * 128 + (threadIdx.x >> 4);
    float v[8][8];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        load8<XT, VEC>(x + (r < rows ? r : rows - 1) * ldx, c, cols, v[i]);
        m = fmaxf(m, max8(v[i]));   // a repeated last row does not change the maximum
    }
#pragma unroll
    for (int o = 32; o; o >>= 1)
        m = fmaxf(m, __shfl_xor(m, o, 64));
    if ((threadIdx.x & 63) == 0)
        top[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const float s = fp8_scale(m, pow2);
    if (threadIdx.x == 0)
        scales[blockIdx.x] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        if (r < rows)
            store8(q + r * ldq, c, cols, v[i], s, pow2, vecq);
    }
}

template <typename XT>
static int launch_quant_t(const XT *x, int64_t ldx, int64_t rows, int cols, int block, bool pow2,
                          uint8_t *q, int64_t ldq, float *scales, hipStream_t s)
{
    const bool vec = ((uintptr_t)x % 16 == 0) && (ldx * (int64_t)sizeof(XT)) % 16 == 0;
    const bool vecq = ((uintptr_t)q % 8 == 0) && ldq % 8 == 0;
    const int64_t nb = (cols + 127) / 128;
    // a launch has fewer than 2^32 threads: rows beyond that take another
    const int64_t most = (1LL << 24) - 1;
    const int64_t step = block == 1 ? most * 16 / nb : most / nb * 128;
#define MOE_Q(KERN, V)                                                                         \
    hipLaunchKernelGGL((KERN<XT, V>), dim3((unsigned)grid), dim3(256), 0, s, x, ldx, n, cols,  \
                       pow2, q, ldq, scales, vecq)
    while (rows > 0) {
        const int64_t n = std::min(rows, step);
        const int64_t grid = block == 1 ? (n * nb + 15) / 16 : (n + 127) / 128 * nb;
        if (block == 1) {
            if (vec) MOE_Q(quant_rows_kernel, true);
            else MOE_Q(quant_rows_kernel, false);
        } else {
            if (vec) MOE_Q(quant_blocks_kernel, true);
            else MOE_Q(quant_blocks_kernel, false);
        }
        MOE_LAUNCH_CHECK("quantisation kernel");
        rows -= n;
        x += n * ldx;
        q += n * ldq;
        scales += (n + block - 1) / block * nb;
    }
#undef MOE_Q
    return MOE_OK;
}

int launch_quant_fp8(const void *x, int dtype, int64_t ldx, int64_t rows, int cols, int block,
                     bool pow2, void *q, int64_t ldq, float *scales, hipStream_t s)
{
    uint8_t *qb = static_cast<uint8_t *>(q);
    if (dtype == MOE_DTYPE_F32)
        return launch_quant_t(static_cast<const float *>(x), ldx, rows, cols, block, pow2, qb, ldq,
                              scales, s);
    if (dtype == MOE_DTYPE_F16)
        return launch_quant_t(static_cast<const f16 *>(x), ldx, rows, cols, block, pow2, qb, ldq,
                              scales, s);
    return launch_quant_t(static_cast<const uint16_t *>(x), ldx, rows, cols, block, pow2, qb, ldq,
                          scales, s);
}

// Before the routed experts' tile kernels, in one launch: the tokens to e4m3
// (power-of-two scales; cols a multiple of 64), and in the last workgroup the
// table of row tiles of at most bm rows, experts in order.  E <= 1024.
__global__ __launch_bounds__(256) void fp8_tokens_kernel(
    const f16 *__restrict__ x, int64_t rows, int cols, uint8_t *__restrict__ q,
    float *__restrict__ scales, const int32_t *__restrict__ offsets,
    const void *const *__restrict__ blobs, int E, int bm, Fp8TileRec *__restrict__ tiles)
{
    if (blockIdx.x == gridDim.x - 1) {
        __shared__ int wsum[4];
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        int o[5], c[4], n = 0;   // thread t: experts 4t..4t+3
#pragma unroll
        for (int i = 0; i < 5; ++i)
            o[i] = offsets[min((int)threadIdx.x * 4 + i, E)];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = (o[i + 1] - o[i] + bm - 1) / bm;
            n += c[i];
        }
        int incl = n;
#pragma unroll
        for (int st = 1; st < 64; st <<= 1) {
            const int v = __shfl_up(incl, st, 64);
            if (lane >= st)
                incl += v;
        }
        if (lane == 63)
            wsum[wave] = incl;
        __syncthreads();
        int at = incl - n;
        for (int i = 0; i < wave; ++i)
            at += wsum[i];
        if (threadIdx.x == 255)
            tiles[0] = Fp8TileRec{nullptr, 0, at + n};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!c[i])
                continue;
            const uint8_t *b = static_cast<const uint8_t *>(blobs[threadIdx.x * 4 + i]);
            for (int j = 0; j < c[i]; ++j)
                tiles[1 + at++] =
                    Fp8TileRec{b, o[i] + j * bm, min(bm, o[i + 1] - o[i] - j * bm)};
        }
        return;
    }
    const int nb = (cols + 127) / 128;
    const int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4;
    if (b >= rows * nb)
        return;
    const int64_t r = b / nb;
    const int kb = (int)(b - r * nb);
    const int c = kb * 128 + (threadIdx.x & 15) * 8;
    float v[8];
    load8<f16, true>(x + r * cols, c, cols, v);
    const float s = fp8_scale(row16_max(max8(v)), true);
    if ((threadIdx.x & 15) == 0)
        scales[b] = s;
    store8(q + r * cols, c, cols, v, s, true, true);
}

int launch_fp8_tokens(const void *x, int64_t rows, int cols, uint8_t *q, float *scales,
                      const int32_t *offsets, const void *const *blobs, int E, int bm,
                      Fp8TileRec *tiles, hipStream_t s)
{
    const int64_t blocks = rows * ((cols + 127) / 128), grid = (blocks + 15) / 16 + 1;
    if (blocks > FP8_MOST_TOKEN_BLOCKS)
        return set_error(MOE_EUNSUPPORTED, "FP8 experts: %lld token blocks, at most %d",
                         (long long)blocks, FP8_MOST_TOKEN_BLOCKS);
    hipLaunchKernelGGL(fp8_tokens_kernel, dim3((unsigned)grid), dim3(256), 0, s,
                       static_cast<const f16 *>(x), rows, cols, q, scales, offsets, blobs, E, bm,
                       tiles);
    MOE_LAUNCH_CHECK("fp8_tokens_kernel");
    return MOE_OK;
}

}  // namespace moe
