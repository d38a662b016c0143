// k_linear.hip -- fp16 matrix products with bias, activation and residual in their
// epilogue, and their gradients: choice of the tiles (k_linear_tile.hip), dz and the
// bias gradient.
//
//   z = x w^T + bias,  out = residual + act(z)
//   dz = dy act'(z),   dx = dz w,   dw = dz^T x,   dbias = sum_m dz
#include <algorithm>

#include "k_linear.h"

namespace moe {

// The forms of a tile: rows, columns, groups that share its k, workgroups a compute
// unit; and what they were measured to take, in us (fp16, K from 256 to 5632, 256
// compute units busy with one to eight workgroups each): a workgroup `end` for its
// first loads and its results and `one` for a block of 64 k (of its group, where
// groups share k); two workgroups on a compute unit together `two` for a block of each.
// The smallest form reads 64 bytes at a time of a b whose rows run across k, and takes
// `across` for a block then; it is not used where a is such too (32 bytes at a time: 64 x
// 2048 x 4096 14.4 us, 32-row tiles in four parts 11.0).
//
// With them the form and the parts of k that take the least time are chosen, among those
// whose workgroups a launch holds.  On 90 products from 1 x 1024 x 256 to 8192 x 8192 x
// 8192 the choice was the fastest form or within 8% of it.  These times are of the kernel
// alone on the same operands again and again, on one card, and tell the forms apart; a
// call on changing inputs takes up to a tenth more (4096 x 11264 x 2048: 163 us on the
// same, 174 to 179 on changing ones; 16 x 5632 x 2048 7.4 and 9.0).  (At K = 2048, chosen / next best: 16 x 5632 16-row tiles 7.4 us,
// 32-row 7.6; 333 x 1408 32-row 8.2, 64-row 9.0; 256 x 5632 64-row 13.7, 128-row
// 17.3; 2048 x 2048 128-row of eight waves 20.8, of four 26.8; 4096 x 2048 the other
// way round, 35.7 and 39.8; 4096 x 5632 192-row 86, 256-row 95; 4096 x 11264 256-row
// 154, 192-row 163; at K = 5632 64 x 2048 16-row 9.7, 32-row in four parts 11.1, 4096
// x 2048 256 x 128 90, 128-row 94).
struct LinForm {
    int bm, bn, kg, per_cu;
    double end, one, two, across;
};
static const LinForm FORMS[] = {
    {16, 32, 8, 1, 3.0, 0.50, 0, 0.80},      {32, 64, 2, 1, 2.2, 0.30, 0, 0.30},
    {64, 64, 2, 1, 2.2, 0.44, 0, 0.44},      {64, 64, 1, 2, 0.9, 0.33, 0.33, 0.33},
    {128, 128, 1, 1, 3.5, 0.50, 0, 0.50},    {128, 128, 1, 2, 1.8, 0.72, 0.90, 0.72},
    {192, 256, 1, 1, 6.0, 1.13, 0, 1.13},    {256, 256, 1, 1, 5.0, 1.45, 0, 1.45},
    {256, 128, 1, 1, 4.4, 0.875, 0, 0.875}};
constexpr int NFORMS = sizeof(FORMS) / sizeof(FORMS[0]);

LinPlan linear_plan(int M, int N, int K, int across)
{
    LinPlan best{0, 1, LIN_MOST_ITEMS + 1};   // (where no form fits a launch)
    double least = 1e300;
    const int nkb = (int)(((int64_t)K + 63) / 64);
    for (int f = 0; f < NFORMS; ++f) {
        const LinForm &o = FORMS[f];
        if (across == 2 && (f == 0 || f == 8))   // (never the fastest there)
            continue;
        const double one = across ? o.across : o.one;
        const int64_t tiles = ((int64_t)M + o.bm - 1) / o.bm * (((int64_t)N + o.bn - 1) / o.bn);
        if (tiles > LIN_MOST_ITEMS)
            continue;
        for (int s = 1; s <= 8; s *= 2) {
            const int each = (nkb + s - 1) / s;
            if (s > 1 && (tiles * s > 256 || (nkb + each - 1) / each != s))
                break;   // no more parts than compute units, none empty
            const int64_t n = (tiles * s + 255) / 256;   // workgroups of a compute unit
            const int64_t pairs = o.per_cu == 2 ? n / 2 : 0;
            const double blocks = (each + o.kg - 1) / o.kg;
            double t = 1.0 + n * o.end + blocks * (pairs * o.two + (n - 2 * pairs) * one);
            if (s > 1)   // a launch more, and the parts' sums written and read
                t += 4.5 + (2.0 * s + 1) * 4.0 * M * N / 3e6;
            if (t < least) {
                least = t;
                best = LinPlan{f, s, tiles * s};
            }
        }
    }
    return best;
}

static size_t plan_ws(const LinPlan &p, int M, int N)
{
    return p.splits == 1 ? 0 : (size_t)p.splits * M * ((N + 7) / 8 * 8) * sizeof(float);
}

LinPlan linear_forward_plan(int M, int N, int K)
{
    if (M > 1 << 30 || N > 1 << 30)
        return LinPlan{0, 1, LIN_MOST_ITEMS + 1};
    return M <= LIN_FEW_ROWS ? LinPlan{0, 1, 1} : linear_plan(M, N, K, 0);
}

size_t linear_ws(const LinPlan &p, int M, int N) { return plan_ws(p, M, N); }

int launch_linear(const LinArgs &a, const LinPlan &p, void *ws, hipStream_t s)
{
    if (a.M <= LIN_FEW_ROWS && !a.a_ks && !a.b_ks)
        return launch_linear_rows(a, s);
    return launch_linear_tile(a, p, ws, s);
}

// ------------------------------------------------------------------ gradients

// dz as the sum of two fp16.  Rounded to one it adds as much to the errors of dx and dw as
// their own rounding (1.41 of it together, among few values by chance much more); as two
// it is off by 2^-21 of itself at most, and they by 1.00.  The products take twice the k
// for it (4096 x 5632 x 2048, SiLU: 400 us), so a caller may ask for one (214).
// Both have dz's sign and neither is zero (but for what fp16's smallest step cannot be
// divided into), so that an infinity in x or w meets no zero and no other sign: hi is the
// last fp16 up to dz, by the conversion towards zero, and lo the rest of up to a step;
// where the rest is zero or rounds to it, hi is the fp16 before and lo the step between
// the two, whose sum is exact.  So they are off by 2^-11 of lo, or by 2^-25.
__device__ __forceinline__ void split_f16(const float (&v)[8], half8_t &hi, half8_t &lo)
{
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const half2_t pair = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_pkrtz(v[j], v[j + 1]));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f16 a = pair[i], b = (f16)(v[j + i] - (float)a);
            if (b == (f16)0.0f && a != (f16)0.0f) {
                const f16 h = a;
                a = __builtin_bit_cast(f16, (uint16_t)(__builtin_bit_cast(uint16_t, h) - 1));
                b = h - a;
            }
            hi[j + i] = a;
            lo[j + i] = __builtin_isinf(a) ? a : b;
        }
    }
}
// Its first `cols` values.
__device__ __forceinline__ void store_half8(f16 *p, int cols, bool vec, half8_t v)
{
    if (vec && cols >= 8) {
        *reinterpret_cast<half8_t *>(p) = v;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cols)
                p[j] = v[j];
    }
}
// A row of dz for dx: its values, then their rests (k starts over in w).  For dw: the
// values, and the rests as the next row (x is taken twice a row); where a row has whole
// pieces of 8 that is the same memory.
struct DzTwo {       // null: one fp16 each
    f16 *row, *col;  // [M][dz, rest] and [M][2][dz or rest]; col null: row's
    int64_t ld_row, ld_col;
};

// dz = dy act'(z) in fp16 (rows of ldd, zeros up to the next multiple of 8 behind
// column N), where dz is not null, and its column sums over `tall` rows, from the
// unrounded values, where parts is not null.  2^lt threads a row, eight columns each.
// 4096 x 5632, SiLU: to one fp16 30 us, bound by memory (4.6 TB/s); to two 51 to 60, the
// splitting and twice the bytes written (184 MB in all, 3.1 to 3.6 TB/s).
template <bool TWO>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinGrads g, f16 *dz, int64_t ldd,
                                                        float *parts, bool vec_y, bool vec_z, int lt, int tall,
                                                        DzTwo two)
{
    __shared__ float sums[256 * 8];   // [row of threads][column]
    const int c = (threadIdx.x & ((1 << lt) - 1)) * 8, rows = 256 >> lt;
    const int n = (blockIdx.x << lt) * 8 + c;
    const int64_t m0 = (int64_t)blockIdx.y * tall;
    const int cols = g.N - n;
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = threadIdx.x >> lt; i < tall; i += rows) {
        const int64_t m = m0 + i;
        if (m >= g.M || cols <= 0)
            break;
        float v[8];
        load_piece<f16, 8>(g.dy + m * g.lddy + n, 0, cols, vec_y, v);
        if (g.act != MOE_ACT_NONE) {
            float z[8];
            load_piece<f16, 8>(g.z + m * g.ldz + n, 0, cols, vec_z, z);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = j < cols ? v[j] * act_grad(z[j], g.act) : 0.0f;
        }
        if (!TWO && dz)
            store_piece<f16, 8>(dz + m * ldd + n, 0, 8, true, v);
        if constexpr (TWO) {
            half8_t hi, lo;
            split_f16(v, hi, lo);
            const bool vec = g.N % 8 == 0;
            store_half8(two.row + m * two.ld_row + n, cols, vec, hi);
            store_half8(two.row + m * two.ld_row + g.N + n, cols, vec, lo);
            if (two.col) {
                store_half8(two.col + 2 * m * two.ld_col + n, 8, true, hi);
                store_half8(two.col + (2 * m + 1) * two.ld_col + n, 8, true, lo);
            }
            if (n + 8 >= g.N)   // zeros up to the next multiple of 8
                for (int64_t k = 2 * (int64_t)g.N; k < two.ld_row; ++k)
                    two.row[m * two.ld_row + k] = (f16)0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] += v[j];
    }
    if (!parts)
        return;
    const int width = 8 << lt;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sums[(threadIdx.x >> lt) * width + c + j] = s[j];
    __syncthreads();
    for (int i = threadIdx.x; i < width; i += 256) {
        const int k = (blockIdx.x << lt) * 8 + i;
        float v = sums[i];
        for (int r = 1; r < rows; ++r)
            v += sums[r * width + i];
        if (k < g.N)
            parts[(int64_t)blockIdx.y * g.N + k] = v;
    }
}

__global__ __launch_bounds__(1024) void linear_dbias_kernel(LinColumns c)
{
    __shared__ float s[16][64];
    column_sums<16>(c, blockIdx.x, s);
}

// Zeros into rows of `cols` elements, ld apart.
template <typename T>
__global__ __launch_bounds__(256) void zero_rows_kernel(T *p, int64_t ld, int64_t rows, int cols)
{
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < rows * cols; i += gridDim.x * 256LL)
        p[i / cols * ld + i % cols] = (T)0.0f;
}

// Rows of a workgroup of linear_dz_kernel: in up to 512 parts, whose sums one more
// workgroup for 64 columns adds up.
static int dz_rows(int M)
{
    const int64_t each = ((int64_t)M + 511) / 512;
    return (int)(each < 64 ? 64 : each);
}
static int dz_groups(int M) { return (M + dz_rows(M) - 1) / dz_rows(M); }
static int64_t dz_ld(int N) { return ((int64_t)N + 7) / 8 * 8; }

LinGradPlan linear_grad_plan(int M, int N, int K)
{
    LinGradPlan p{};
    if (M > 1 << 30 || K > 1 << 30 || N > LIN_MOST_LD)
        return p;
    p.dx = linear_plan(M, K, N, 1);
    p.dw = linear_plan(N, K, M, 2);
    p.fits = p.dx.items <= LIN_MOST_ITEMS && p.dw.items <= LIN_MOST_ITEMS;
    if (M <= LIN_MOST_TWICE) {
        p.dx2 = linear_plan(M, K, 2 * N, 1);
        p.dw2 = linear_plan(N, K, 2 * M, 2);
        p.fits2 = p.dx2.items <= LIN_MOST_ITEMS && p.dw2.items <= LIN_MOST_ITEMS;
    }
    size_t most = std::max(plan_ws(p.dx, M, K), plan_ws(p.dw, N, K));
    if (p.fits2)
        most = std::max({most, plan_ws(p.dx2, M, K), plan_ws(p.dw2, N, K)});
    p.col = al256((int64_t)M * dz_ld(p.fits2 ? 2 * N : N) * 2);
    p.parts = p.col + (p.fits2 && N % 8 ? al256(2 * (int64_t)M * dz_ld(N) * 2) : 0);
    p.products = p.parts + al256((int64_t)dz_groups(M) * N * 4);
    p.total = p.products + (int64_t)most;
    return p;
}

int launch_linear_backward(const LinGrads &g, const LinGradPlan &w, void *ws, hipStream_t s)
{
    if (g.M == 0) {
        if (g.dbias) {
            hipLaunchKernelGGL(linear_dbias_kernel, dim3((g.N + 63) / 64), dim3(1024), 0, s,
                               LinColumns{nullptr, 0, g.N, g.dbias});
            MOE_LAUNCH_CHECK("linear_dbias_kernel");
        }
        if (g.dw) {
            const unsigned grid =
                (unsigned)std::min<int64_t>(((int64_t)g.N * g.K + 255) / 256, 4096);
            if (g.odt == MOE_DTYPE_F32)
                hipLaunchKernelGGL(zero_rows_kernel<float>, dim3(grid), dim3(256), 0, s,
                                   static_cast<float *>(g.dw), g.lddw, (int64_t)g.N, g.K);
            else
                hipLaunchKernelGGL(zero_rows_kernel<f16>, dim3(grid), dim3(256), 0, s,
                                   static_cast<f16 *>(g.dw), g.lddw, (int64_t)g.N, g.K);
            MOE_LAUNCH_CHECK("zero_rows_kernel");
        }
        return MOE_OK;
    }
    uint8_t *base = static_cast<uint8_t *>(ws);
    float *parts = reinterpret_cast<float *>(base + w.parts);
    // dy itself is dz where nothing changes it and its rows end on whole pieces
    const bool own = g.act != MOE_ACT_NONE || g.N % 8 || g.lddy % 8 || (uintptr_t)g.dy % 16 ||
                     g.lddy > LIN_MOST_LD;
    const bool two = g.two && (g.dx || g.dw);
    const DzTwo rest = {two ? static_cast<f16 *>(ws) : nullptr,
                        g.N % 8 ? reinterpret_cast<f16 *>(base + w.col) : nullptr, dz_ld(2 * g.N),
                        dz_ld(g.N)};
    const LinPlan &dx = two ? w.dx2 : w.dx, &dw = two ? w.dw2 : w.dw;
    const f16 *dz = own ? static_cast<const f16 *>(ws) : g.dy;
    const int64_t ldd = own ? dz_ld(g.N) : g.lddy;
    const int G = dz_groups(g.M);
    const LinColumns cols = {parts, G, g.N, g.dbias};
    // the bias gradient's last step joins the launch that joins dw's parts, if there is one
    const bool late = g.dw && dw.splits > 1;
    if ((own && (g.dx || g.dw)) || g.dbias) {
        int lt = 0;   // threads of a row: up to 32
        while (lt < 5 && (8 << lt) < g.N)
            ++lt;
        auto rows16 = [](const void *p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; };
        hipLaunchKernelGGL(two ? linear_dz_kernel<true> : linear_dz_kernel<false>,
                           dim3((g.N + (8 << lt) - 1) / (8 << lt), G), dim3(256), 0, s, g,
                           own && (g.dx || g.dw) ? static_cast<f16 *>(ws) : nullptr, ldd,
                           g.dbias ? parts : nullptr, rows16(g.dy, g.lddy), rows16(g.z, g.ldz), lt,
                           dz_rows(g.M), rest);
        MOE_LAUNCH_CHECK("linear_dz_kernel");
        if (g.dbias && !late) {
            hipLaunchKernelGGL(linear_dbias_kernel, dim3((g.N + 63) / 64), dim3(1024), 0, s, cols);
            MOE_LAUNCH_CHECK("linear_dbias_kernel");
        }
    }
    LinArgs a{};
    a.act = MOE_ACT_NONE;
    a.odt = g.odt;
    a.a = dz;
    a.lda = ldd;
    a.b_ks = true;
    a.N = g.K;
    if (g.dx) {
        a.b = g.w;
        a.ldb = g.ldw;
        a.M = g.M;
        a.K = g.N;
        if (two) {
            a.lda = rest.ld_row;
            a.K = 2 * g.N;
            a.twice = true;
        }
        a.out = g.dx;
        a.ldo = g.lddx;
        const int rc = launch_linear(a, dx, base + w.products, s);
        if (rc)
            return rc;
    }
    if (g.dw) {
        a.a_ks = true;
        a.b = g.x;
        a.ldb = g.ldx;
        a.M = g.N;
        a.K = g.M;
        if (two) {
            a.a = rest.col ? rest.col : rest.row;
            a.lda = rest.ld_col;
            a.K = 2 * g.M;
            a.twice = true;
        }
        a.out = g.dw;
        a.ldo = g.lddw;
        if (g.dbias && late)
            a.columns = cols;
        return launch_linear(a, dw, base + w.products, s);
    }
    return MOE_OK;
}

}  // namespace moe
