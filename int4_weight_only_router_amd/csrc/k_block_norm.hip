// k_block_norm.hip -- the end of one block and the start of the next:
//
//   u = post(y) or y,   r = residual + scale * gate * u,   n = pre(r)
//
// with RMS or layer norms, and its gradients.  One pass: a row stays in fp32
// registers from its loads to its stores, so every value is read once and
// written once, and n is formed from the unrounded r.  A layer norm's variance
// is the mean square of the centred values (a second sum over registers), not a
// difference of two large means.  Bound by memory: 4096 x 2048 fp16 with both norms and
// a shared gate 15.1 us, 4.4 TB/s of the 4.9 that a copy reaches; one row 2.3 us.
#include <algorithm>

#include "k_block.h"

namespace moe {

// One value of a row, zero past its end (`at` in bytes).
template <typename T>
__device__ __forceinline__ float row_load(__amdgpu_buffer_rsrc_t r, int at)
{
    if constexpr (sizeof(T) == 4)
        return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
    else
        return (float)__builtin_bit_cast(
            T, (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0));
}
template <typename T>
__device__ __forceinline__ void row_store(__amdgpu_buffer_rsrc_t r, int at, float v)
{
    if constexpr (sizeof(T) == 4)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, at, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)v), r, at, 0, 0);
}

// Eight values in a row of H (a multiple of 8), 16 bytes at a time.
template <typename T>
__device__ __forceinline__ void row_load8(__amdgpu_buffer_rsrc_t r, int at, float (&v)[8])
{
    if constexpr (sizeof(T) == 4) {
        const float4_t a = __builtin_bit_cast(float4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
        const float4_t b =
            __builtin_bit_cast(float4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16, 0, 0));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
        typedef typename Vec8<T>::type V;
        const V a = __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)a[j];
    }
}
template <typename T>
__device__ __forceinline__ void row_store8(__amdgpu_buffer_rsrc_t r, int at, const float (&v)[8])
{
    if constexpr (sizeof(T) == 4) {
        const float4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uint4_t, a), r, at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uint4_t, b), r, at + 16, 0, 0);
    } else {
        typename Vec8<T>::type a;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            a[j] = (T)v[j];
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uint4_t, a), r, at, 0, 0);
    }
}

// The columns of a row among its threads.  VEC: chunk i of a thread is eight
// columns in a row (16 bytes of fp16).  Otherwise (odd sizes, strides or addresses)
// eight columns `span` apart, so that a wave's loads are contiguous all the same.
// Rows are the same for a whole wave.
template <bool VEC>
struct Cols {
    int t, span, H;   // thread of the row, threads of a row, columns
    __device__ __forceinline__ int col(int i, int j) const
    {
        return VEC ? (i * span + t) * 8 + j : (i * 8 + j) * span + t;
    }
    // (The column is formed anew at each use: kept, the places and masks of a thread's
    // columns take the registers of its values.)
    __device__ __forceinline__ int fresh(int i, int j) const
    {
        int k = t;
        asm volatile("" : "+v"(k));
        return VEC ? (i * span + k) * 8 + j : (i * 8 + j) * span + k;
    }
    __device__ __forceinline__ bool in(int i, int j) const
    {
        return (VEC ? col(i, 0) : fresh(i, j)) < H;
    }
    template <typename T>
    __device__ __forceinline__ void load(const T *row, int i, float (&v)[8]) const
    {
        if constexpr (VEC) {
            row_load8<T>(row_rsrc(row, H), col(i, 0) * (int)sizeof(T), v);
        } else {
            const __amdgpu_buffer_rsrc_t r = row_rsrc(row, H);
            const int k = fresh(i, 0);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = row_load<T>(r, (k + j * span) * (int)sizeof(T));
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *row, int i, const float (&v)[8]) const
    {
        if constexpr (VEC) {
            row_store8<T>(row_rsrc(row, H), col(i, 0) * (int)sizeof(T), v);
        } else {
            const __amdgpu_buffer_rsrc_t r = row_rsrc(row, H);
            const int k = fresh(i, 0);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                row_store<T>(r, (k + j * span) * (int)sizeof(T), v[j]);
        }
    }
    // weights: fp32 or of the rows' type
    template <typename T>
    __device__ __forceinline__ void weights(const void *w, bool w32, int i, float (&v)[8]) const
    {
        if (sizeof(T) == 4 || w32)
            load<float>(static_cast<const float *>(w), i, v);
        else
            load<T>(static_cast<const T *>(w), i, v);
    }
};

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
template <int W, int NC, bool VEC>
__device__ __forceinline__ void normalise(float (&v)[NC][8], const Cols<VEC> &c, const NormArgs &a,
                                          float *part, int &half)
{
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
                v[i][j] = c.in(i, j) ? v[i][j] - mean : 0.0f;
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
template <typename XT, int NC, bool VEC>
__device__ __forceinline__ void affine(float (&v)[NC][8], const Cols<VEC> &c, const NormArgs &a,
                                       const void *w, const void *b)
{
    const float one = a.offset ? 1.0f : 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float t[8];
        if (w) {
            c.template weights<XT>(w, a.w32, i, t);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] *= t[j] + one;
        }
        if (b) {
            c.template weights<XT>(b, a.w32, i, t);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] += t[j];
        }
    }
}

// W waves a row of up to 512 W NC columns: a wave a row (no barrier, all its
// loads in flight together) up to 2048 columns, above that, and for few rows, the
// workgroup (333 x 1000 bf16, layer norms, odd stride: 5.4 us, a wave a row 16.6).
template <typename XT, bool VEC, int W, int NC>
__global__ __launch_bounds__(256) void block_norm_kernel(NormArgs a)
{
    __shared__ float part[2 * W];
    constexpr int ROWS = 4 / W;
    const Cols<VEC> c = {W == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x, 64 * W, a.H};
    int half = 0;
    const int64_t t = (int64_t)blockIdx.x * ROWS +
                      (W == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0);
    if (t < a.T) {   // (the whole row's threads)
        float r[NC][8], u[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (a.residual) {
                c.load(static_cast<const XT *>(a.residual) + t * a.ldr, i, r[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    r[i][j] = 0.0f;
            }
        }
        if (a.y) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                c.load(static_cast<const XT *>(a.y) + t * a.ldy, i, u[i]);
            if (a.post) {
                normalise<W, NC>(u, c, a, part, half);
                affine<XT>(u, c, a, a.post_w, a.post_b);
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                if (a.gate) {
                    float g[8];
                    c.load(static_cast<const XT *>(a.gate) + t * a.ldg, i, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        u[i][j] *= g[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    r[i][j] = __builtin_fmaf(a.scale, u[i][j], r[i][j]);
            }
        }
        if (a.out) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                c.store(static_cast<XT *>(a.out) + t * a.ldo, i, r[i]);
        }
        if (a.n) {
            normalise<W, NC>(r, c, a, part, half);
            affine<XT>(r, c, a, a.pre_w, a.pre_b);
#pragma unroll
            for (int i = 0; i < NC; ++i)
                c.store(static_cast<XT *>(a.n) + t * a.ldn, i, r[i]);
        }
    }
}

template <typename XT, bool VEC>
static int launch_norm_t(const NormArgs &a, hipStream_t s)
{
    // a wave a row where rows alone give every SIMD (1024) one
    const bool wave = a.H <= 512 || (a.H <= 2048 && a.T >= 1024);
    const int rows = wave ? 4 : 1;   // of a workgroup
    const int64_t grid = ((int64_t)a.T + rows - 1) / rows;
#define MOE_N(W, NC)                                                                             \
    hipLaunchKernelGGL((block_norm_kernel<XT, VEC, W, NC>), dim3((unsigned)grid), dim3(256), 0, s, \
                       a)
    if (wave && a.H <= 512) MOE_N(1, 1);
    else if (wave && a.H <= 1024) MOE_N(1, 2);
    else if (wave) MOE_N(1, 4);
    else if (a.H <= 2048) MOE_N(4, 1);
    else if (a.H <= 4096) MOE_N(4, 2);
    else MOE_N(4, 4);
#undef MOE_N
    MOE_LAUNCH_CHECK("block_norm_kernel");
    return MOE_OK;
}

template <typename XT>
static int launch_norm_x(NormArgs a, hipStream_t s)
{
    // a launch has fewer than 2^32 threads: rows beyond that take another
    const int64_t most = (1 << 23), s1 = sizeof(XT);
    auto on = [&](const void *p, int64_t ld) {
        return p ? static_cast<const char *>(p) + most * ld * s1 : nullptr;
    };
    for (int64_t left = a.T; left > 0; left -= most) {
        a.T = (int)std::min(left, most);
        const int rc = a.vec ? launch_norm_t<XT, true>(a, s) : launch_norm_t<XT, false>(a, s);
        if (rc)
            return rc;
        a.y = on(a.y, a.ldy);
        a.residual = on(a.residual, a.ldr);
        a.gate = on(a.gate, a.ldg);
        a.out = const_cast<char *>(on(a.out, a.ldo));
        a.n = const_cast<char *>(on(a.n, a.ldn));
    }
    return MOE_OK;
}

int launch_block_norm(const NormArgs &a, int dtype, hipStream_t s)
{
    if (dtype == MOE_DTYPE_F32)
        return launch_norm_x<float>(a, s);
    return dtype == MOE_DTYPE_F16 ? launch_norm_x<f16>(a, s) : launch_norm_x<bf16>(a, s);
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
//
// 4096 x 2048 fp16, both norms, shared gate (100 MB of rows): 30.3 us and 4.8 for the
// sums, 34 a call.  Four waves a SIMD (registers: three sums of eight columns and six
// rows' values) issue 468 vector instructions a row and wave, half of the time, and
// meet at a barrier for each of the row's four sums; reading the next rows ahead took
// 3.4 us off, fewer instructions 4.3.  No more rows fit: twice the workgroups would
// write twice the 12.6 MB of partial sums.

typedef float float2v_t __attribute__((ext_vector_type(2)));
constexpr int NB_THREADS = 512, NB_WAVES = NB_THREADS / 64;
enum { NB_GATE = 0, NB_POST_W, NB_POST_B, NB_PRE_W, NB_PRE_B, NB_SUMS };

// LDS accesses while direct-to-LDS loads are in flight: without a restrict pointer the
// compiler takes them to alias those loads and waits for them.
template <typename T>
__device__ __forceinline__ T lds_get(const T *__restrict__ p) { return *p; }
template <typename T>
__device__ __forceinline__ void lds_put(T *__restrict__ p, T v) { *p = v; }

// Sums over a row's W waves (groups of W waves in a row) of a and, with `two`, of b.
__device__ __forceinline__ void group_sum(float &a, float &b, bool two, int W, float2v_t *part,
                                          int &half)
{
    a = wave_sum_f32(a);
    if (two)
        b = wave_sum_f32(b);
    if (W == 1)
        return;
    const int wave = threadIdx.x >> 6;
    float2v_t *p = part + half * NB_WAVES;
    half ^= 1;
    if ((threadIdx.x & 63) == 0)
        lds_put(p + wave, float2v_t{a, b});
    lds_barrier();
    const int w0 = wave & ~(W - 1);
    float2v_t v = lds_get(p + w0);
    for (int i = 1; i < W; ++i) {
        const float2v_t o = lds_get(p + w0 + i);
        v.x += o.x;
        v.y += o.y;
    }
    a = v.x;
    b = v.y;
}

// 1 / sqrt(v) by the hardware's reciprocal root (an ulp); values below its range are
// scaled into it.
__device__ __forceinline__ float recip_root(float v)
{
    const bool low = v < 0x1p-100f;
    return __builtin_amdgcn_rsqf(low ? v * 0x1p100f : v) * (low ? 0x1p50f : 1.0f);
}

// v to its normalised values; returns the reciprocal root (0 for a turn past the
// last row, whose zeros must stay zeros also where eps is 0).
template <int NC, bool VEC>
__device__ __forceinline__ float normalise_group(float (&v)[NC][8], const Cols<VEC> &c, bool live,
                                                 const NormArgs &a, float per_h, int W,
                                                 float2v_t *part, int &half)
{
    float s = 0.0f, none = 0.0f;
    if (a.layer) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += v[i][j];
        group_sum(s, none, false, W, part, half);
        const float mean = s * per_h;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = c.in(i, j) ? v[i][j] - mean : 0.0f;
        s = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s = __builtin_fmaf(v[i][j], v[i][j], s);
    group_sum(s, none, false, W, part, half);
    const float rho = live ? recip_root(__builtin_fmaf(s, per_h, a.eps)) : 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[i][j] *= rho;
    return rho;
}

// g = dn * w to the gradient of the normed row (zeros past its end); m its normalised
// values.
template <int NC, bool VEC>
__device__ __forceinline__ void norm_input_grad(float (&g)[NC][8], const float (&m)[NC][8],
                                                const Cols<VEC> &c, float rho, const NormArgs &a,
                                                float per_h, int W, float2v_t *part, int &half)
{
    float s = 0.0f, q = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q = __builtin_fmaf(g[i][j], m[i][j], q);
    if (a.layer) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += g[i][j];
    }
    group_sum(q, s, a.layer, W, part, half);
    const float along = q * per_h * rho;
    if (a.layer) {
        const float mean = s * per_h;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                g[i][j] = c.in(i, j) ? g[i][j] - mean : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            g[i][j] = __builtin_fmaf(-m[i][j], along, rho * g[i][j]);
}

// v *= a weight; weight(i, t): its values in columns i
template <int NC, typename F>
__device__ __forceinline__ void times_weight(float (&v)[NC][8], F &&weight)
{
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float t[8];
        weight(i, t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[i][j] *= t[j];
    }
}

// Floats from one workgroup's sums to the next one's: a memory channel's run more than
// they are, since H is often a multiple of all channels' and their reader's loads would
// meet on one (H = 2048: 12.0 us instead of 4.6 with 16 loads in flight).
__host__ __device__ constexpr int64_t nb_pitch(int n, int H) { return (int64_t)n * H + 64; }

// LDS of a workgroup: the row sums' halves, the biases' sums (each thread's in places
// of its own), and behind them, AHEAD, a piece a thread of every tensor's next row and
// the weights; where those stood the groups meet at the end.
constexpr int NB_PART = 2 * NB_WAVES * sizeof(float2v_t), NB_PIECES = NB_THREADS * 16;
constexpr int NB_COLS = NB_THREADS * 8 * sizeof(float);
static int norm_backward_lds(const NormArgs &a, const NormGrads &d, int W, bool ahead)
{
    const int nc = a.H > 512 * W ? 2 : 1;
    const int biases = (d.sums[NB_POST_B] != nullptr) + (d.sums[NB_PRE_B] != nullptr);
    const int rows = (a.y != nullptr) + (a.residual != nullptr) + (d.dn != nullptr) +
                     (d.dout != nullptr) + (a.gate != nullptr);
    const int weights = a.post + (a.post_b != nullptr) + 1;
    const int next = ahead ? rows * NB_PIECES + weights * W * 512 * (int)sizeof(float) : 0;
    return NB_PART + biases * nc * NB_COLS + std::max(next, NB_COLS);
}

// NC: eights of columns of a thread (W waves hold 512 W NC).  The sums of the biases'
// gradients are seldom asked for; they stand in LDS and leave the registers to the
// others.  AHEAD (16-bit rows): the next turn's rows travel to LDS while this turn is
// computed, each thread's piece to its own place, so no barrier is needed for them;
// the weights (ones for absent ones) stand in LDS too, as loads behind those would
// wait for them.
template <typename XT, bool VEC, int NC, bool AHEAD>
__global__ __launch_bounds__(NB_THREADS, NC == 1 ? 4 : 2) void block_norm_backward_kernel(
    NormArgs a, NormGrads d, int W)
{
    static_assert(!AHEAD || (VEC && NC == 1 && sizeof(XT) == 2), "a piece is 16 bytes");
    extern __shared__ __align__(16) unsigned char nb_smem[];
    float2v_t *part = reinterpret_cast<float2v_t *>(nb_smem);
    typedef float Places[NB_THREADS];   // of one sum
    Places *post_bias = reinterpret_cast<Places *>(nb_smem + NB_PART);
    Places *pre_bias = post_bias + (d.sums[NB_POST_B] ? NC * 8 : 0);
    float *cols = reinterpret_cast<float *>(pre_bias + (d.sums[NB_PRE_B] ? NC * 8 : 0));
    const int groups = NB_WAVES / W;   // rows at a time
    const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / W;
    const int H = a.H;
    const float per_h = 1.0f / (float)H;
    Cols<VEC> c = {(int)threadIdx.x - grp * W * 64, 64 * W, H};
    int half = 0;
    float sum[NB_SUMS][NC][8];
    const bool post_b = d.sums[NB_POST_B], pre_b = d.sums[NB_PRE_B];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum[NB_GATE][i][j] = sum[NB_POST_W][i][j] = sum[NB_PRE_W][i][j] = 0.0f;
            if (post_b)
                post_bias[i * 8 + j][threadIdx.x] = 0.0f;
            if (pre_b)
                pre_bias[i * 8 + j][threadIdx.x] = 0.0f;
        }
    // AHEAD: the pieces of y, residual, dn, dout and gate, then the weights
    unsigned char *pieces = reinterpret_cast<unsigned char *>(cols);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    auto each_row = [&](int64_t t, auto &&f) {   // f(number of the tensor, its row)
        auto row = [&](const void *p, int64_t ld) { return static_cast<const XT *>(p) + t * ld; };
        int n = 0;
        if (a.y)
            f(n++, row(a.y, a.ldy));
        if (a.residual)
            f(n++, row(a.residual, a.ldr));
        if (d.dn)
            f(n++, row(d.dn, a.ldn));
        if (d.dout)
            f(n++, row(d.dout, a.ldo));
        if (a.gate)
            f(n++, row(a.gate, a.ldg));
    };
    auto send = [&](int64_t t0) {   // the rows of a turn on their way
        const int at = c.t * 8 < H ? c.t * 8 : 0;
        each_row(t0 + grp < a.T ? t0 + grp : 0, [&](int n, const XT *row) {
            dma16(row + at, pieces + n * NB_PIECES + wave * 1024);
        });
        asm volatile("" ::: "memory");
    };
    const float *lds_w[3];   // post_w, post_b, pre_w
    if constexpr (AHEAD) {
        send((int64_t)blockIdx.x * groups);
        int rows = 0;
        each_row(0, [&](int, const XT *) { ++rows; });
        float *to = reinterpret_cast<float *>(pieces + rows * NB_PIECES);
        const void *from[3] = {a.post_w, a.post_b, a.pre_w};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            lds_w[k] = to;
            if (k == 1 ? !a.post_b : k == 0 && !a.post)
                continue;
            const float one = k != 1 && (a.offset || !from[k]) ? 1.0f : 0.0f;
            for (int i = threadIdx.x; i < W * 512; i += NB_THREADS) {
                float w = 0.0f;
                if (from[k] && i < H)
                    w = a.w32 ? static_cast<const float *>(from[k])[i]
                              : (float)static_cast<const XT *>(from[k])[i];
                to[i] = w + one;
            }
            to += W * 512;
        }
        wait_vm<0>();
        __syncthreads();
    }
    auto weight = [&](int k, const void *w, int i, float (&v)[8]) {
        if constexpr (AHEAD) {
            const float4_t *p = reinterpret_cast<const float4_t *>(lds_w[k] + c.t * 8);
            const float4_t lo = lds_get(p), hi = lds_get(p + 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = lo[j];
                v[4 + j] = hi[j];
            }
        } else {
            c.template weights<XT>(w, a.w32, i, v);
            const float one = a.offset && k != 1 ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] += one;
        }
    };
    auto bump = [](float *p, float v) { lds_put(p, lds_get(p) + v); };
    // stores of a turn, which stand behind the next turn's loads
    const int stores = (d.dresidual != nullptr) +
                       (a.y ? (d.dgate && a.ldg) + (d.dy != nullptr) : 0);
    const int64_t turn = (int64_t)gridDim.x * groups;
    // every group takes as many turns (its sums meet at barriers); one past the
    // last row works on zeros and stores nothing
    for (int64_t t0 = (int64_t)blockIdx.x * groups; t0 < a.T; t0 += turn) {
        // (the weights are read again every turn, out of the caches: kept, they would
        // take the registers of the sums)
        if constexpr (!AHEAD)
            asm volatile("" : "+s"(a.post_w), "+s"(a.post_b), "+s"(a.pre_w));
        const bool live = t0 + grp < a.T;
        const int64_t t = live ? t0 + grp : 0;
        c.H = live ? H : 0;   // columns that this turn may touch
        float u[NC][8], r[NC][8], gate[NC][8], pm[NC][8], dr[NC][8], g[NC][8];
        float post_rho = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                u[i][j] = r[i][j] = dr[i][j] = g[i][j] = 0.0f;
            if (!a.gate)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    gate[i][j] = 1.0f;
            auto load = [&](int n, const void *p, int64_t ld, float (&v)[8]) {
                if constexpr (AHEAD) {
                    typedef typename Vec8<XT>::type V;
                    const uint4_t p = *reinterpret_cast<const uint4_t *>(
                        pieces + n * NB_PIECES + threadIdx.x * 16);
                    const V x = __builtin_bit_cast(V, p & (c.t * 8 < c.H ? ~0u : 0u));
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = (float)x[j];
                } else {
                    c.load(static_cast<const XT *>(p) + t * ld, i, v);
                }
            };
            int n = 0;
            if (a.y)
                load(n++, a.y, a.ldy, u[i]);
            if (a.residual)
                load(n++, a.residual, a.ldr, r[i]);
            if (d.dn)
                load(n++, d.dn, a.ldn, g[i]);
            if (d.dout)
                load(n++, d.dout, a.ldo, dr[i]);
            if (a.gate)
                load(n++, a.gate, a.ldg, gate[i]);
        }
        const bool more = t0 + turn < a.T;
        if constexpr (AHEAD) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the pieces are read
            if (more)
                send(t0 + turn);
        }
        if (a.y) {
            if (a.post) {
                post_rho = normalise_group(u, c, live, a, per_h, W, part, half);
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        pm[i][j] = u[i][j];
                if (AHEAD || a.post_w)
                    times_weight(u, [&](int i, float (&v)[8]) { weight(0, a.post_w, i, v); });
                if (a.post_b)
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        float w[8];
                        weight(1, a.post_b, i, w);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            u[i][j] += w[j];
                    }
            }
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    r[i][j] = __builtin_fmaf(a.scale, gate[i][j] * u[i][j], r[i][j]);
        }
        if (d.dn) {
            const float rho = normalise_group(r, c, live, a, per_h, W, part, half);   // r: normalised
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sum[NB_PRE_W][i][j] = __builtin_fmaf(g[i][j], r[i][j], sum[NB_PRE_W][i][j]);
                    if (pre_b)
                        bump(&pre_bias[i * 8 + j][threadIdx.x], g[i][j]);
                }
            if (AHEAD || a.pre_w)
                times_weight(g, [&](int i, float (&v)[8]) { weight(2, a.pre_w, i, v); });
            norm_input_grad(g, r, c, rho, a, per_h, W, part, half);
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dr[i][j] += g[i][j];
        }
        if (d.dresidual)
#pragma unroll
            for (int i = 0; i < NC; ++i)
                c.store(static_cast<XT *>(d.dresidual) + t * a.ldr, i, dr[i]);
        if (a.y) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dr[i][j] *= a.scale;                                 // of gate * u
                    u[i][j] *= dr[i][j];                                 // the gate's
                    sum[NB_GATE][i][j] += u[i][j];
                    dr[i][j] *= gate[i][j];                              // of u
                }
                if (d.dgate && a.ldg)
                    c.store(static_cast<XT *>(d.dgate) + t * a.ldg, i, u[i]);
            }
            if (a.post) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        sum[NB_POST_W][i][j] = __builtin_fmaf(dr[i][j], pm[i][j], sum[NB_POST_W][i][j]);
                        if (post_b)
                            bump(&post_bias[i * 8 + j][threadIdx.x], dr[i][j]);
                    }
                if (AHEAD || a.post_w)
                    times_weight(dr, [&](int i, float (&v)[8]) { weight(0, a.post_w, i, v); });
                norm_input_grad(dr, pm, c, post_rho, a, per_h, W, part, half);
            }
            if (d.dy)
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    c.store(static_cast<XT *>(d.dy) + t * a.ldy, i, dr[i]);
        }
        if (AHEAD && more) {   // the next rows are there, if not yet this turn's stores
            if (stores == 3)
                wait_vm<3>();
            else if (stores == 2)
                wait_vm<2>();
            else if (stores == 1)
                wait_vm<1>();
            else
                wait_vm<0>();
        }
    }
    if constexpr (AHEAD)
        __syncthreads();   // the weights' places are the groups' from here
    // the groups' sums, in the order of the groups
    c.H = H;
    float *to = d.parts + blockIdx.x * nb_pitch(d.nsums, H);
#pragma unroll
    for (int k = 0; k < NB_SUMS; ++k) {
        if (!d.sums[k])
            continue;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (k == NB_POST_B || k == NB_PRE_B)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sum[k][i][j] = (k == NB_PRE_B ? pre_bias : post_bias)[i * 8 + j][threadIdx.x];
            if (groups > 1) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    cols[j * NB_THREADS + threadIdx.x] = sum[k][i][j];
                __syncthreads();
                if (grp == 0)
                    for (int o = 1; o < groups; ++o)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            sum[k][i][j] += cols[j * NB_THREADS + o * W * 64 + threadIdx.x];
            }
            if (grp == 0)
                c.store(to, i, sum[k][i]);
        }
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
    const int64_t pitch = nb_pitch(to.n, H);
    float v = 0.0f;
    if (col < H) {
#pragma unroll 16
        for (int g = wave; g < G; g += 16)
            v += parts[g * pitch + blockIdx.y * (int64_t)H + col];
    }
    s[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && col < H) {
#pragma unroll
        for (int i = 1; i < 16; ++i)
            v += s[i][lane];
        to.p[blockIdx.y][col] = v;
    }
}

// Waves a row: the fewest (a power of two, up to a workgroup's) that hold H columns,
// eight a lane; rows of more than 4096 columns take 16 a lane.
static int norm_waves(int H)
{
    int w = 1;
    while (w * 512 < H && w < NB_WAVES)
        w *= 2;
    return w;
}

constexpr int NB_GRID = 512;   // two workgroups a compute unit
static int norm_backward_grid(int T, int H)
{
    const int rows = NB_WAVES / norm_waves(H);
    return (int)std::min<int64_t>(((int64_t)T + rows - 1) / rows, NB_GRID);
}

size_t block_norm_backward_ws(int T, int H)
{
    return (size_t)(norm_backward_grid(T, H) * nb_pitch(NB_SUMS, H)) * sizeof(float);
}

template <typename XT, bool VEC, int NC, bool AHEAD>
static int launch_backward_t(const NormArgs &a, const NormGrads &d, int G, int W, hipStream_t s)
{
    static LdsLimit limit;
    const int rc = limit.raise((const void *)block_norm_backward_kernel<XT, VEC, NC, AHEAD>,
                               160 * 1024);
    if (rc)
        return rc;
    hipLaunchKernelGGL((block_norm_backward_kernel<XT, VEC, NC, AHEAD>), dim3((unsigned)G),
                       dim3(NB_THREADS), norm_backward_lds(a, d, W, AHEAD), s, a, d, W);
    MOE_LAUNCH_CHECK("block_norm_backward_kernel");
    return MOE_OK;
}

template <typename XT>
static int launch_backward_x(const NormArgs &a, const NormGrads &d, int G, int W, hipStream_t s)
{
    if (a.H > 512 * NB_WAVES)
        return a.vec ? launch_backward_t<XT, true, 2, false>(a, d, G, W, s)
                     : launch_backward_t<XT, false, 2, false>(a, d, G, W, s);
    if constexpr (sizeof(XT) == 2)   // ahead where LDS holds two workgroups all the same
        if (a.vec && norm_backward_lds(a, d, W, true) <= 80 * 1024)
            return launch_backward_t<XT, true, 1, true>(a, d, G, W, s);
    return a.vec ? launch_backward_t<XT, true, 1, false>(a, d, G, W, s)
                 : launch_backward_t<XT, false, 1, false>(a, d, G, W, s);
}

int launch_block_norm_backward(const NormArgs &a, NormGrads d, int dtype, hipStream_t s)
{
    const int W = norm_waves(a.H), G = norm_backward_grid(a.T, a.H);
    NormSums to{};
    for (int k = 0; k < NB_SUMS; ++k)
        if (d.sums[k])
            to.p[to.n++] = d.sums[k];
    d.nsums = to.n;
    if (a.T > 0) {
        const int rc = dtype == MOE_DTYPE_F32   ? launch_backward_x<float>(a, d, G, W, s)
                       : dtype == MOE_DTYPE_F16 ? launch_backward_x<f16>(a, d, G, W, s)
                                                : launch_backward_x<bf16>(a, d, G, W, s);
        if (rc)
            return rc;
    }
    if (to.n) {   // without tokens: zeros
        hipLaunchKernelGGL(norm_sums_kernel, dim3((a.H + 63) / 64, to.n), dim3(1024), 0, s,
                           d.parts, G, a.H, to);
        MOE_LAUNCH_CHECK("norm_sums_kernel");
    }
    return MOE_OK;
}

}  // namespace moe
