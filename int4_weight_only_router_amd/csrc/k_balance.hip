// k_balance.hip -- balance loss and z loss of router logits, per-expert counts,
// and the gradient of the logits.
//
// Over the n unmasked tokens, with p the scores divided by their sum:
//   counts_e  choices of e,  f_e = counts_e / sum counts,  P_e = 1/n sum_t p_te
//   balance = coef E sum_e f_e P_e,   z = zcoef / n sum_t lse_t^2
//   dbalance/dl_te = coef / n p_te (d_e - sum_j p_tj d_j) [(1 - s_te) for sigmoid scores]
//   dz/dl_te = zcoef / n 2 lse_t softmax_te
// with d_e = E f_e - 1: p sums to one, so the one drops out, and with it the
// cancellation of a load that is nearly even (d_e is formed from whole numbers).
// The counts are needed before any gradient, the logits only once: a wave takes a
// row, holds it in registers and writes its gradient at once.
//
// A sigmoid score's ratio is formed as a_e / sum a with a_e = exp(min(l_e, 0) - m)
// / (1 + exp(-|l_e|)) and m the row's largest min(l, 0), so that it does not
// underflow where every logit is far below zero.
#include <algorithm>

#include "k_balance.h"

namespace moe {

constexpr int BL_THREADS = 256, BL_WAVES = BL_THREADS / 64;
constexpr int BL_ONE_THREADS = 1024;

template <typename T>
__device__ __forceinline__ float logit_value(T v)
{
    const float f = (float)v;
    // NaN counts as masked, +inf as the largest finite value (as in the selection)
    return f == f ? fminf(f, 3.402823466e+38f) : -__builtin_inff();
}

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int o = 32; o; o >>= 1)
        v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}

// Choices and unmasked tokens of the tokens t0 <= t < t1 into hist (LDS [E]) and
// the return value (this thread's share).
__device__ __forceinline__ int count_tokens(const BalanceArgs &a, int64_t t0, int64_t t1, int *hist,
                                            int threads)
{
    int n = 0;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += threads)
        n += !a.mask || a.mask[t];
    if (a.idx)
        for (int64_t i = t0 * a.k + threadIdx.x; i < t1 * a.k; i += threads)
            if (!a.mask || a.mask[i / a.k]) {
                const int e = a.idx[i];
                if ((unsigned)e < (unsigned)a.E)
                    atomicAdd(&hist[e], 1);
            }
    return n;
}

// Sum over the workgroup (every thread gets it); s: one int a wave.
__device__ __forceinline__ int block_sum(int v, int *s, int waves)
{
#pragma unroll
    for (int o = 32; o; o >>= 1)
        v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0)
        s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < waves; ++i)
        v += s[i];
    __syncthreads();
    return v;
}

// One row: its p into p[], its share of the balance loss and lse^2 added up, its
// gradient written.  Lane l holds experts l, l + 64, ...
template <typename LT, int NE>
__device__ __forceinline__ void balance_row(const BalanceArgs &a, int64_t t, const float (&d)[NE],
                                            float per_n, float up, float (&psum)[NE], float &loss,
                                            float &zsum)
{
    const int lane = threadIdx.x & 63;
    const bool on = !a.mask || a.mask[t];
    if (!on && !a.dlogits)
        return;
    const LT *row = static_cast<const LT *>(a.logits) + t * a.ld;
    float l[NE], p[NE], top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        l[i] = on && e < a.E ? logit_value<LT>(row[e]) : -__builtin_inff();
        top = fmaxf(top, l[i]);
    }
    top = wave_max(top);
    const bool some = top > -__builtin_inff();   // not masked throughout
    const bool sig = a.score == MOE_SCORE_SIGMOID;
    const float zc = a.zcoef * per_n;
    float lse = 0.0f, inv_soft = 0.0f;
    if (some && (!sig || a.zcoef != 0.0f)) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            p[i] = expf(l[i] - top);
            s += p[i];
        }
        s = wave_sum_f32(s);
        lse = top + logf(s);
        inv_soft = 1.0f / s;
    }
    float dot = 0.0f, share = 0.0f;
    float part[NE];   // p (softmax: without its 1/s factor until below)
    if (sig) {
        const float m = fminf(top, 0.0f);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            part[i] = some ? expf(fminf(l[i], 0.0f) - m) / (1.0f + expf(-fabsf(l[i]))) : 0.0f;
            s += part[i];
        }
        s = wave_sum_f32(s);
        const float inv = some ? 1.0f / s : 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            part[i] *= inv;
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            part[i] = some ? p[i] * inv_soft : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        psum[i] += part[i];
        dot = __builtin_fmaf(part[i], d[i], dot);
        share += part[i];
    }
    dot = wave_sum_f32(dot);
    loss += dot + wave_sum_f32(share);   // sum p (d + 1)
    if (a.zcoef != 0.0f)
        zsum = __builtin_fmaf(lse, lse, zsum);
    if (!a.dlogits)
        return;
    const float cb = up * a.coef * per_n, cz = up * zc * 2.0f * lse * inv_soft;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        float g = cb * part[i] * (d[i] - dot);
        if (sig) {   // 1 - sigmoid(l)
            const float x = expf(-fabsf(l[i]));
            g *= (l[i] > 0.0f ? x : 1.0f) / (1.0f + x);
        }
        if (a.zcoef != 0.0f && some)
            g = __builtin_fmaf(cz, p[i], g);
        if (e < a.E) {
            g = on ? g : 0.0f;
            const int64_t at = t * a.ldd + e;
            if (a.gtype == MOE_DTYPE_F32)
                static_cast<float *>(a.dlogits)[at] = g;
            else if (a.gtype == MOE_DTYPE_F16)
                static_cast<f16 *>(a.dlogits)[at] = (f16)g;
            else
                static_cast<__bf16 *>(a.dlogits)[at] = (__bf16)g;
        }
    }
}

// d_e of this lane's experts from whole counts.
template <int NE>
__device__ __forceinline__ void deviations(const int *hist, int64_t total, int E, float (&d)[NE])
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        d[i] = e < E ? (float)((double)(hist[e] * (int64_t)E - total) /
                               (double)(total > 0 ? total : 1))
                     : 0.0f;
    }
}

__device__ __forceinline__ int64_t total_choices(const int *hist, int E)
{
    int64_t s = 0;   // every wave for itself
    for (int e = threadIdx.x & 63; e < E; e += 64)
        s += hist[e];
#pragma unroll
    for (int o = 32; o; o >>= 1)
        s += __shfl_xor(s, o, 64);
    return s;
}

// Partial counts of the tokens dealt out over the workgroups: [G][E] and the
// unmasked tokens [G].
__global__ __launch_bounds__(BL_ONE_THREADS) void balance_count_kernel(BalanceArgs a)
{
    __shared__ int hist[BL_MAX_E];
    __shared__ int s[BL_ONE_THREADS / 64];
    for (int e = threadIdx.x; e < a.E; e += BL_ONE_THREADS)
        hist[e] = 0;
    __syncthreads();
    const int64_t each = ((int64_t)a.T + gridDim.x - 1) / gridDim.x;
    const int64_t t0 = blockIdx.x * each;
    const int n = block_sum(count_tokens(a, t0, min(t0 + each, (int64_t)a.T), hist, BL_ONE_THREADS),
                            s, BL_ONE_THREADS / 64);
    for (int e = threadIdx.x; e < a.E; e += BL_ONE_THREADS)
        a.part_counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
    if (threadIdx.x == 0)
        a.part_n[blockIdx.x] = n;
}

// Rows: partial sums of p [G][E], of the balance loss and of lse^2 [G][2].
template <typename LT, int NE>
__global__ __launch_bounds__(BL_THREADS) void balance_rows_kernel(BalanceArgs a)
{
    __shared__ int hist[64 * NE];
    __shared__ float cols[BL_WAVES][64 * NE + 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < a.E; e += BL_THREADS) {
        int c = 0;
        if (a.idx)
            for (int g = 0; g < a.count_groups; ++g)
                c += a.part_counts[(int64_t)g * a.E + e];
        else
            c = a.counts[e];
        hist[e] = c;
    }
    int64_t n = a.T;
    if (a.mask) {
        n = 0;
        for (int g = 0; g < a.count_groups; ++g)
            n += a.part_n[g];
    }
    __syncthreads();
    float d[NE], psum[NE], loss = 0.0f, zsum = 0.0f;
    deviations<NE>(hist, total_choices(hist, a.E), a.E, d);
#pragma unroll
    for (int i = 0; i < NE; ++i)
        psum[i] = 0.0f;
    const float per_n = n > 0 ? 1.0f / (float)n : 0.0f;
    const float up = a.dlogits && a.d_loss ? *a.d_loss : 1.0f;
    for (int64_t t = (int64_t)blockIdx.x * BL_WAVES + wave; t < a.T;
         t += (int64_t)gridDim.x * BL_WAVES)
        balance_row<LT, NE>(a, t, d, per_n, up, psum, loss, zsum);
#pragma unroll
    for (int i = 0; i < NE; ++i)
        cols[wave][lane + 64 * i] = psum[i];
    if (lane == 0) {
        cols[wave][64 * NE] = loss;
        cols[wave][64 * NE + 1] = zsum;
    }
    __syncthreads();
    float *to = a.part_p + (int64_t)blockIdx.x * (a.E + 2);
    for (int e = threadIdx.x; e < a.E + 2; e += BL_THREADS) {
        const int at = e < a.E ? e : 64 * NE + e - a.E;
        to[e] = (cols[0][at] + cols[1][at]) + (cols[2][at] + cols[3][at]);
    }
}

// The outputs from the partial sums: 64 experts a workgroup, 16 partial sums at a
// time; workgroup 0 also the losses.
__global__ __launch_bounds__(BL_ONE_THREADS) void balance_join_kernel(BalanceArgs a, int G)
{
    __shared__ float s[16][64];
    __shared__ int si[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 64 + lane;
    int64_t n = a.T;
    if (a.mask) {
        n = 0;
        for (int g = 0; g < a.count_groups; ++g)
            n += a.part_n[g];
    }
    const double per_n = n > 0 ? 1.0 / (double)n : 0.0;
    float v = 0.0f;
    int c = 0;
    if (e < a.E) {
        for (int g = wave; g < G; g += 16)
            v += a.part_p[(int64_t)g * (a.E + 2) + e];
        if (a.idx)
            for (int g = wave; g < a.count_groups; g += 16)
                c += a.part_counts[(int64_t)g * a.E + e];
    }
    s[wave][lane] = v;
    si[wave][lane] = c;
    __syncthreads();
    if (wave == 0 && e < a.E) {
        for (int i = 1; i < 16; ++i) {
            v += s[i][lane];
            c += si[i][lane];
        }
        if (a.mean_prob)
            a.mean_prob[e] = (float)(v * per_n);
        if (a.idx)
            a.counts[e] = c;
    }
    if (blockIdx.x == 0 && wave == 1 && a.losses) {
        double b = 0.0, z = 0.0;
        for (int g = lane; g < G; g += 64) {
            b += a.part_p[(int64_t)g * (a.E + 2) + a.E];
            z += a.part_p[(int64_t)g * (a.E + 2) + a.E + 1];
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            b += __shfl_xor(b, o, 64);
            z += __shfl_xor(z, o, 64);
        }
        if (lane == 0) {
            a.losses[0] = (float)(a.coef * b * per_n);
            a.losses[1] = a.zcoef != 0.0f ? (float)(a.zcoef * z * per_n) : 0.0f;
        }
    }
}

// Few tokens: all of it in one workgroup.
template <typename LT, int NE>
__global__ __launch_bounds__(BL_ONE_THREADS) void balance_one_kernel(BalanceArgs a)
{
    constexpr int WAVES = BL_ONE_THREADS / 64;
    __shared__ int hist[64 * NE];
    __shared__ int s[WAVES];
    __shared__ float cols[WAVES][64 * NE + 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < a.E; e += BL_ONE_THREADS)
        hist[e] = a.idx ? 0 : a.counts[e];
    __syncthreads();
    const int n = block_sum(count_tokens(a, 0, a.T, hist, BL_ONE_THREADS), s, WAVES);
    float d[NE], psum[NE], loss = 0.0f, zsum = 0.0f;
    deviations<NE>(hist, total_choices(hist, a.E), a.E, d);
#pragma unroll
    for (int i = 0; i < NE; ++i)
        psum[i] = 0.0f;
    const float per_n = n > 0 ? 1.0f / (float)n : 0.0f;
    const float up = a.dlogits && a.d_loss ? *a.d_loss : 1.0f;
    for (int t = wave; t < a.T; t += WAVES)
        balance_row<LT, NE>(a, t, d, per_n, up, psum, loss, zsum);
#pragma unroll
    for (int i = 0; i < NE; ++i)
        cols[wave][lane + 64 * i] = psum[i];
    if (lane == 0) {
        cols[wave][64 * NE] = loss;
        cols[wave][64 * NE + 1] = zsum;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E + 2; e += BL_ONE_THREADS) {
        const int at = e < a.E ? e : 64 * NE + e - a.E;
        float v = 0.0f;
        for (int w = 0; w < WAVES; ++w)
            v += cols[w][at];
        v *= per_n;
        if (e < a.E) {
            if (a.mean_prob)
                a.mean_prob[e] = v;
            if (a.idx)
                a.counts[e] = hist[e];
        } else if (a.losses) {
            a.losses[e - a.E] = e == a.E ? a.coef * v : a.zcoef != 0.0f ? a.zcoef * v : 0.0f;
        }
    }
}

// No tokens: zeros.
__global__ void balance_none_kernel(BalanceArgs a)
{
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        if (a.mean_prob)
            a.mean_prob[e] = 0.0f;
        a.counts[e] = 0;
    }
    if (a.losses && threadIdx.x < 2)
        a.losses[threadIdx.x] = 0.0f;
}

constexpr int BL_ONE_ROWS = 64;   // rows up to which one workgroup does it all
constexpr int BL_COUNT_GROUPS = 16, BL_GROUPS = 512;

static int count_groups(int T) { return std::min((T + 255) / 256, BL_COUNT_GROUPS); }
static int row_groups(int T) { return std::min((T + BL_WAVES - 1) / BL_WAVES, BL_GROUPS); }

size_t balance_ws(int T, int E)
{
    if (T <= BL_ONE_ROWS)
        return 0;
    return (size_t)al256((int64_t)count_groups(T) * (E + 1) * 4) +
           (size_t)row_groups(T) * (E + 2) * 4;
}

template <typename LT, int NE>
static int launch_ne(const BalanceArgs &a, hipStream_t s)
{
    if (a.T <= BL_ONE_ROWS) {
        hipLaunchKernelGGL((balance_one_kernel<LT, NE>), dim3(1), dim3(BL_ONE_THREADS), 0, s, a);
        MOE_LAUNCH_CHECK("balance_one_kernel");
        return MOE_OK;
    }
    if (a.idx || a.mask) {
        hipLaunchKernelGGL(balance_count_kernel, dim3(a.count_groups), dim3(BL_ONE_THREADS), 0, s, a);
        MOE_LAUNCH_CHECK("balance_count_kernel");
    }
    const int G = row_groups(a.T);
    hipLaunchKernelGGL((balance_rows_kernel<LT, NE>), dim3(G), dim3(BL_THREADS), 0, s, a);
    MOE_LAUNCH_CHECK("balance_rows_kernel");
    hipLaunchKernelGGL(balance_join_kernel, dim3((a.E + 63) / 64), dim3(BL_ONE_THREADS), 0, s, a, G);
    MOE_LAUNCH_CHECK("balance_join_kernel");
    return MOE_OK;
}

template <typename LT>
static int launch_type(const BalanceArgs &a, hipStream_t s)
{
    if (a.E <= 64) return launch_ne<LT, 1>(a, s);
    if (a.E <= 128) return launch_ne<LT, 2>(a, s);
    if (a.E <= 256) return launch_ne<LT, 4>(a, s);
    if (a.E <= 512) return launch_ne<LT, 8>(a, s);
    return launch_ne<LT, 16>(a, s);
}

int launch_balance(BalanceArgs a, int dtype, void *ws, hipStream_t s)
{
    if (a.T == 0) {
        hipLaunchKernelGGL(balance_none_kernel, dim3(1), dim3(256), 0, s, a);
        MOE_LAUNCH_CHECK("balance_none_kernel");
        return MOE_OK;
    }
    a.count_groups = count_groups(a.T);
    uint8_t *base = static_cast<uint8_t *>(ws);
    a.part_counts = reinterpret_cast<int *>(base);
    a.part_n = a.part_counts + (int64_t)a.count_groups * a.E;
    a.part_p = reinterpret_cast<float *>(base + al256((int64_t)a.count_groups * (a.E + 1) * 4));
    if (dtype == MOE_DTYPE_F32)
        return launch_type<float>(a, s);
    return dtype == MOE_DTYPE_F16 ? launch_type<f16>(a, s) : launch_type<__bf16>(a, s);
}

}  // namespace moe
