// k_balance.hip -- balance loss and z loss of router logits, per-expert counts,
// and the gradient of the logits.
//
// Over the n unmasked tokens, with p the scores divided by their sum:
//   counts_e  choices of e,  f_e = counts_e / sum counts,  P_e = 1/n sum_t p_te
//   balance = coef E sum_e f_e P_e,   z = zcoef / n sum_t lse_t^2
//   dbalance/dl_te = coef / n p_te (d_e - sum_j p_tj d_j) [(1 - s_te) for sigmoid scores]
//   dz/dl_te = zcoef / n 2 lse_t softmax_te
// with d_e = E f_e - 1: p sums to one, so the one drops out, and with it the
// cancellation of a load that is nearly even (d_e is formed from whole numbers).  The
// loss itself is the sum of E f_e P_e, whose terms are positive: formed from the d_e it
// would cancel where the load lies on unlikely experts, and count a load of zero as even.
// The counts are needed before any gradient, the logits only once: a wave takes a
// row, holds it in registers and writes its gradient at once.
//
// A sigmoid score's ratio is formed as a_e / sum a with a_e = exp(min(l_e, 0) - m) /
// (1 + exp(-|l_e|)) and m the row's largest min(l, 0) where that is far below zero,
// so that it does not underflow where every logit is.
//
// Launches: up to 64 tokens one workgroup does it all (16 x 64: 4.4 us); else the rows (a
// wave each, 16 waves a workgroup, sums of p over them to the workspace) and the joining
// of their sums, and before them the counts where every workgroup counting all choices
// for itself would take longer.  Bound by the launches and their dependent steps: 4096 x
// 512 with sigmoid scores, z loss and gradient 15.5 us, of which the counts 3.8, the
// rows 10.2 (17 MB, 1.7 TB/s; half of it vector instructions, 760 a row), the
// joining 3.5.
#include <algorithm>

#include "k_balance.h"
#include "k_block.h"

namespace moe {

constexpr int BL_THREADS = 1024, BL_WAVES = BL_THREADS / 64;
// Waves of a workgroup of rows: half as many where a lane holds 16 experts (registers).
template <int NE>
constexpr int bl_waves() { return NE > 8 ? 8 : 16; }
constexpr int BL_ONE_ROWS = 64;   // tokens up to which one workgroup does it all
// Choices up to which every workgroup counts all of them for itself (eight a thread:
// 1 us, against 2 to 3 of another launch), else in up to 16 workgroups of a launch.
constexpr int BL_SELF = 8192;
constexpr int BL_COUNT_GROUPS = 16, BL_GROUPS = 256;
constexpr float BL_FAR = -60.0f;   // exp(-60) and its sums are far inside fp32's range

// NaN counts as masked, +inf as the largest finite value (as in the selection)
__device__ __forceinline__ float logit_value(float f)
{
    return fminf(fmaxf(f, -__builtin_inff()), 3.402823466e+38f);
}

// exp(x) for x <= 0 by the hardware's exp2 (an ulp), with the rounding of x log2(e)
// made good: 0 far below fp32's range and for -inf.
__device__ __forceinline__ float exp_neg(float x)
{
    constexpr float L2E = 1.4426950408889634f, L2E_LO = 1.9259629911266175e-8f;
    const float t = fmaxf(x, -200.0f) * L2E;
    const float r = __builtin_fmaf(fmaxf(x, -200.0f), L2E, -t) + fmaxf(x, -200.0f) * L2E_LO;
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e * r, 0.69314718055994531f, e);
}

template <int CTRL>
__device__ __forceinline__ float dpp_max_step(float v)
{
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                                  0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false)));
}
__device__ __forceinline__ float wave_max(float v)
{
    v = dpp_max_step<0xB1>(v);    // the steps of wave_sum_f32
    v = dpp_max_step<0x4E>(v);
    v = dpp_max_step<0x141>(v);
    v = dpp_max_step<0x140>(v);
    const int i = __builtin_bit_cast(int, v);
    auto row = [&](int lane) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(i, lane));
    };
    return fmaxf(fmaxf(row(0), row(16)), fmaxf(row(32), row(48)));
}

// Choices and unmasked tokens of the tokens t0 <= t < t1 into hist (LDS [E]) and
// the return value (this thread's share).  (T k < 2^31; a choice and its token's mask
// are loaded together, several of them before the first is counted.)
template <int THREADS>
__device__ __forceinline__ int count_tokens(const BalanceArgs &a, int t0, int t1, int *hist)
{
    int n = 0;
    if (a.mask)
        for (int64_t t = t0 + (int)threadIdx.x; t < t1; t += THREADS)
            n += a.mask[t] != 0;
    if (!a.idx)
        return n;
    constexpr int U = 4;
    const unsigned i1 = (unsigned)t1 * a.k, k = a.k;
    for (unsigned i0 = (unsigned)t0 * k + threadIdx.x; i0 < i1; i0 += U * THREADS) {
        int e[U];
        uint8_t on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned i = min(i0 + u * THREADS, i1 - 1);
            e[u] = a.idx[i];
            on[u] = a.mask ? a.mask[i / k] : 1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * THREADS < i1 && (unsigned)e[u] < (unsigned)a.E && on[u])
                atomicAdd(&hist[e[u]], 1);
    }
    return n;
}

__device__ __forceinline__ int wave_sum_int(int v)
{
#pragma unroll
    for (int o = 32; o; o >>= 1)
        v += __shfl_xor(v, o, 64);
    return v;
}
// (16 bits and the rest are sums of whole numbers below 2^24, so exact in fp32)
__device__ __forceinline__ int64_t wave_sum_counts(int64_t v)
{
    return (int64_t)wave_sum_f32((float)(v & 0xffff)) +
           ((int64_t)wave_sum_f32((float)(v >> 16)) << 16);
}

// A row's logits and its token's mask in registers, as they were loaded: lane l holds
// experts l, l + 64, ...  (Nothing here waits for them.)
template <typename LT, int NE>
struct Row {
    LT v[NE];
    uint8_t mask;
    __device__ __forceinline__ void load(const BalanceArgs &a, int64_t t)
    {
        const __amdgpu_buffer_rsrc_t r = row_rsrc(static_cast<const LT *>(a.logits) + t * a.ld, a.E);
        mask = a.mask ? a.mask[t] : 1;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int at = ((int)(threadIdx.x & 63) + 64 * i) * (int)sizeof(LT);
            if constexpr (sizeof(LT) == 4)
                v[i] = __builtin_bit_cast(LT, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
            else
                v[i] = __builtin_bit_cast(
                    LT, (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0));
        }
    }
    // the logits (-inf past E and for a masked token), and whether the token counts
    __device__ __forceinline__ bool values(const BalanceArgs &a, float (&l)[NE]) const
    {
        const bool on = __builtin_amdgcn_readfirstlane(mask);   // (the same for the whole wave)
        const int E = on ? a.E : 0;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            l[i] = (int)(threadIdx.x & 63) + 64 * i < E ? logit_value((float)v[i])
                                                      : -__builtin_inff();
        return on;
    }
};

template <int NE, typename T>
__device__ __forceinline__ void store_row(const BalanceArgs &a, int64_t t, const float (&g)[NE])
{
    const __amdgpu_buffer_rsrc_t r = row_rsrc(static_cast<T *>(a.dlogits) + t * a.ldd, a.E);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int at = ((int)(threadIdx.x & 63) + 64 * i) * (int)sizeof(T);
        if constexpr (sizeof(T) == 4)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, g[i]), r, at, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)g[i]), r, at, 0, 0);
    }
}

// The row: its p added to psum[], its lse^2 to zsum, its gradient written.
template <int NE>
__device__ __forceinline__ void balance_row(const BalanceArgs &a, int64_t t,
                                            const float (&l)[NE], const float (&d)[NE], float per_n,
                                            float up, float (&psum)[NE], float &zsum)
{
    float top = l[0];
#pragma unroll
    for (int i = 1; i < NE; ++i)
        top = fmaxf(top, l[i]);
    top = wave_max(top);
    const bool some = top > -__builtin_inff();   // not masked throughout
    const bool sig = a.score == MOE_SCORE_SIGMOID;
    float soft[NE], p[NE], lse = 0.0f;
    if (some && (!sig || a.zcoef != 0.0f)) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            soft[i] = exp_neg(l[i] - top);
            s += soft[i];
        }
        s = wave_sum_f32(s);
        lse = top + __logf(s);
        const float inv = 1.0f / s;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            soft[i] *= inv;
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            soft[i] = 0.0f;
    }
    float rest[NE];   // sigmoid scores: 1 - s
    if (sig) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float x = exp_neg(-fabsf(l[i])), q = __builtin_amdgcn_rcpf(1.0f + x);
            const bool up = l[i] > 0.0f;
            rest[i] = up ? x * q : q;
            p[i] = up ? q : x * q;
        }
        if (top < BL_FAR) {   // (all of them far below zero: rest is one)
#pragma unroll
            for (int i = 0; i < NE; ++i)
                p[i] = some ? exp_neg(l[i] - top) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < NE; ++i)
            s += p[i];
        s = wave_sum_f32(s);
        const float inv = some ? 1.0f / s : 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            p[i] *= inv;
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            p[i] = soft[i];
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        psum[i] += p[i];
        dot = __builtin_fmaf(p[i], d[i], dot);
    }
    zsum = __builtin_fmaf(lse, lse, zsum);
    if (!a.dlogits)
        return;
    dot = wave_sum_f32(dot);
    const float cb = up * a.coef * per_n, cz = a.zcoef != 0.0f ? up * a.zcoef * per_n * 2.0f : 0.0f;
    float g[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i)
        g[i] = cb * p[i] * (d[i] - dot);
    if (sig)
#pragma unroll
        for (int i = 0; i < NE; ++i)
            g[i] *= rest[i];
    // (zeros for masked experts and tokens, also where up is not finite; lse times the
    // rest, as by itself it can take cz out of fp32's range)
#pragma unroll
    for (int i = 0; i < NE; ++i)
        g[i] = l[i] > -__builtin_inff() ? __builtin_fmaf(cz * soft[i], lse, g[i]) : 0.0f;
    if (a.gtype == MOE_DTYPE_F32)
        store_row<NE, float>(a, t, g);
    else if (a.gtype == MOE_DTYPE_F16)
        store_row<NE, f16>(a, t, g);
    else
        store_row<NE, __bf16>(a, t, g);
}

// d_e = E f_e - 1 from whole counts.
__device__ __forceinline__ float deviation(int c, int E, int64_t total, float inv)
{
    const bool low = total < 1 << 23 && total * E < 1LL << 31;   // (full-rate products)
    return (low ? (float)(__mul24(c, E) - (int)total) : (float)(c * (int64_t)E - total)) * inv;
}

// Partial counts of the tokens dealt out over the workgroups: [G][E] and the
// unmasked tokens [G].
__global__ __launch_bounds__(BL_THREADS) void balance_count_kernel(BalanceArgs a)
{
    __shared__ int hist[BL_MAX_E];
    __shared__ int s[BL_WAVES];
    for (int e = threadIdx.x; e < a.E; e += BL_THREADS)
        hist[e] = 0;
    __syncthreads();
    const int64_t each = ((int64_t)a.T + gridDim.x - 1) / gridDim.x;
    const int t0 = (int)min(blockIdx.x * each, (int64_t)a.T), t1 = (int)min(t0 + each, (int64_t)a.T);
    const int own = wave_sum_int(count_tokens<BL_THREADS>(a, t0, t1, hist));
    if ((threadIdx.x & 63) == 0)
        s[threadIdx.x >> 6] = own;
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += BL_THREADS)
        a.part_counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
    if (threadIdx.x == 0) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < BL_WAVES; ++i)
            n += s[i];
        a.part_n[blockIdx.x] = n;
    }
}

// Rows.  ONE: of one workgroup, which writes the outputs; else its sums of p, of the
// balance loss and of lse^2 to the workspace [G][E + 2], and workgroup 0 the counts
// and the number of unmasked tokens.
template <typename LT, int NE, bool ONE>
__global__ __launch_bounds__(64 * bl_waves<NE>()) void balance_rows_kernel(BalanceArgs a)
{
    constexpr int WAVES = bl_waves<NE>(), THREADS = 64 * WAVES, HALF = WAVES / 2;
    constexpr int PER = (64 * NE + THREADS - 1) / THREADS;   // experts of a thread
    __shared__ int hist[64 * NE];
    __shared__ float dev[64 * NE];
    __shared__ int64_t totals[WAVES];
    __shared__ int tokens[WAVES];
    __shared__ float cols[HALF][64 * NE + 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t t = (int64_t)blockIdx.x * WAVES + wave;
    // the first row is on its way while the choices are counted
    Row<LT, NE> row;
    row.load(a, t < a.T ? t : 0);
    const float up = a.dlogits && a.d_loss ? *a.d_loss : 1.0f;
    const bool self = ONE || !a.count_groups;   // counts for itself
    int c[PER], own_n = 0;
    if (self) {
        if (a.idx) {
            for (int e = threadIdx.x; e < 64 * NE; e += THREADS)
                hist[e] = 0;
            lds_barrier();
        }
        if (a.idx || a.mask)
            own_n = count_tokens<THREADS>(a, 0, a.T, hist);
        if (a.idx)
            lds_barrier();
    } else if (a.mask && threadIdx.x < a.count_groups) {
        own_n = a.part_n[threadIdx.x];
    }
    int64_t own = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x + i * THREADS;
        c[i] = 0;
        if (e < a.E) {
            if (!a.idx) {
                c[i] = a.counts[e];
            } else if (self) {
                c[i] = hist[e];
            } else {
                int part[BL_COUNT_GROUPS];   // (all on their way together)
#pragma unroll
                for (int g = 0; g < BL_COUNT_GROUPS; ++g)
                    part[g] = a.part_counts[(int64_t)min(g, a.count_groups - 1) * a.E + e];
#pragma unroll
                for (int g = 0; g < BL_COUNT_GROUPS; ++g)
                    c[i] += g < a.count_groups ? part[g] : 0;
            }
        }
        own += c[i];
    }
    own = wave_sum_counts(own);
    if (a.mask)
        own_n = wave_sum_int(own_n);
    if (lane == 0) {
        totals[wave] = own;
        tokens[wave] = own_n;
    }
    lds_barrier();
    int64_t total = 0;
    int n = a.mask ? 0 : a.T;
#pragma unroll
    for (int i = 0; i < WAVES; ++i)
        total += totals[i];
    if (a.mask)
#pragma unroll
        for (int i = 0; i < WAVES; ++i)
            n += tokens[i];
    const float inv = 1.0f / (float)(total > 0 ? total : 1);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x + i * THREADS;
        if (e < 64 * NE) {
            dev[e] = e < a.E ? deviation(c[i], a.E, total, inv) : 0.0f;
            hist[e] = c[i];   // (this thread's own to here)
        }
        if (blockIdx.x == 0 && e < a.E && a.idx)
            a.counts[e] = c[i];
    }
    lds_barrier();
    float d[NE], psum[NE], zsum = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        d[i] = dev[lane + 64 * i];
        psum[i] = 0.0f;
    }
    const float per_n = n > 0 ? 1.0f / (float)n : 0.0f;
    const int64_t step = (int64_t)gridDim.x * WAVES;
    while (t < a.T) {
        float l[NE];
        const bool on = row.values(a, l);
        const int64_t t0 = t;
        t += step;
        if (t < a.T)
            row.load(a, t);
        if (on || a.dlogits)
            balance_row<NE>(a, t0, l, d, per_n, up, psum, zsum);
    }
    float loss = 0.0f;   // sum E f_e p_e of the wave's rows
    const float each = (float)a.E * inv;
#pragma unroll
    for (int i = 0; i < NE; ++i)
        loss = __builtin_fmaf(psum[i], (float)hist[lane + 64 * i] * each, loss);
    loss = wave_sum_f32(loss);
    // the waves' sums: the upper half's onto the lower half's, then those
    if (wave >= HALF) {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            cols[wave - HALF][lane + 64 * i] = psum[i];
        if (lane == 0) {
            cols[wave - HALF][64 * NE] = loss;
            cols[wave - HALF][64 * NE + 1] = zsum;
        }
    }
    lds_barrier();
    if (wave < HALF) {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            cols[wave][lane + 64 * i] += psum[i];
        if (lane == 0) {
            cols[wave][64 * NE] += loss;
            cols[wave][64 * NE + 1] += zsum;
        }
    }
    lds_barrier();
    for (int e = threadIdx.x; e < a.E + 2; e += THREADS) {
        const int at = e < a.E ? e : 64 * NE + e - a.E;
        float v = cols[0][at];
#pragma unroll
        for (int w = 1; w < HALF; ++w)
            v += cols[w][at];
        if (!ONE) {
            a.part_p[(int64_t)blockIdx.x * (a.E + 2) + e] = v;
        } else if (e >= a.E) {
            if (a.losses)
                a.losses[e - a.E] = e > a.E && a.zcoef == 0.0f ? 0.0f
                                    : (e == a.E ? a.coef : a.zcoef) * (v * per_n);
        } else if (a.mean_prob) {
            a.mean_prob[e] = v * per_n;
        }
    }
    if (!ONE && blockIdx.x == 0 && threadIdx.x == 0)
        *a.n = n;
}

// The outputs from the partial sums: 64 experts a workgroup, 16 partial sums at a
// time; the last workgroup the losses.
__global__ __launch_bounds__(BL_THREADS) void balance_join_kernel(BalanceArgs a, int G)
{
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 64 + lane;
    const int n = *a.n;
    const double per_n = n > 0 ? 1.0 / n : 0.0;
    const int64_t ld = a.E + 2;
    if (blockIdx.x == gridDim.x - 1) {
        if (wave > 1 || !a.losses)
            return;
        double v = 0.0;
#pragma unroll 4
        for (int g = lane; g < G; g += 64)
            v += a.part_p[g * ld + a.E + wave];
#pragma unroll
        for (int o = 32; o; o >>= 1)
            v += __shfl_xor(v, o, 64);
        if (lane == 0)
            a.losses[wave] = wave && a.zcoef == 0.0f ? 0.0f
                             : (float)((wave ? a.zcoef : a.coef) * v * per_n);
        return;
    }
    float v = 0.0f;
    if (e < a.E) {
#pragma unroll 16
        for (int g = wave; g < G; g += 16)
            v += a.part_p[g * ld + e];
    }
    s[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && e < a.E) {
#pragma unroll
        for (int i = 1; i < 16; ++i)
            v += s[i][lane];
        if (a.mean_prob)
            a.mean_prob[e] = (float)(v * per_n);
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

// 0: counted by every workgroup.  (Given counts count as few: k = 1.)
static int count_groups(int T, int k)
{
    return (int64_t)T * k <= BL_SELF ? 0 : std::min((int)(((int64_t)T + 255) / 256), BL_COUNT_GROUPS);
}
static int row_groups(int T, int E)
{
    const int waves = E > 512 ? bl_waves<16>() : bl_waves<8>();
    return (int)std::min<int64_t>(((int64_t)T + waves - 1) / waves, BL_GROUPS);
}

size_t balance_ws(int T, int E)
{
    if (T <= BL_ONE_ROWS)
        return 0;
    return (size_t)al256((int64_t)BL_COUNT_GROUPS * (E + 1) * 4 + 4) +
           (size_t)row_groups(T, E) * (E + 2) * 4;
}

template <typename LT, int NE>
static int launch_ne(const BalanceArgs &a, hipStream_t s)
{
    if (a.T <= BL_ONE_ROWS) {
        hipLaunchKernelGGL((balance_rows_kernel<LT, NE, true>), dim3(1), dim3(64 * bl_waves<NE>()), 0, s, a);
        MOE_LAUNCH_CHECK("balance_rows_kernel");
        return MOE_OK;
    }
    if (a.count_groups) {
        hipLaunchKernelGGL(balance_count_kernel, dim3(a.count_groups), dim3(BL_THREADS), 0, s, a);
        MOE_LAUNCH_CHECK("balance_count_kernel");
    }
    const int G = row_groups(a.T, a.E);
    hipLaunchKernelGGL((balance_rows_kernel<LT, NE, false>), dim3(G), dim3(64 * bl_waves<NE>()), 0, s, a);
    MOE_LAUNCH_CHECK("balance_rows_kernel");
    if (a.mean_prob || a.losses) {
        hipLaunchKernelGGL(balance_join_kernel, dim3((a.E + 63) / 64 + 1), dim3(BL_THREADS), 0, s, a,
                           G);
        MOE_LAUNCH_CHECK("balance_join_kernel");
    }
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
    // without choices to count and tokens to leave out there is nothing to count
    a.count_groups = a.idx ? count_groups(a.T, a.k) : a.mask ? count_groups(a.T, 1) : 0;
    uint8_t *base = static_cast<uint8_t *>(ws);
    a.n = reinterpret_cast<int *>(base);
    a.part_counts = a.n + 1;
    a.part_n = a.part_counts + (int64_t)BL_COUNT_GROUPS * a.E;
    a.part_p = reinterpret_cast<float *>(base + al256((int64_t)BL_COUNT_GROUPS * (a.E + 1) * 4 + 4));
    if (dtype == MOE_DTYPE_F32)
        return launch_type<float>(a, s);
    return dtype == MOE_DTYPE_F16 ? launch_type<f16>(a, s) : launch_type<__bf16>(a, s);
}

}  // namespace moe
