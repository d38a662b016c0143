// k_route_select.hip -- expert selection from router logits: softmax or
// sigmoid scores, a selection bias, expert groups, top-k, weights; and the
// router logits of small batches.
//
//   s_e = exp(l_e - max l) / sum_j exp(l_j - max l)   or   1 / (1 + exp(-l_e))
//   c_e = s_e + b_e                                    (decides, does not weigh)
//   G_g = max c over group g, or the sum of its two largest c
//   chosen: the k largest c among the experts of the groups with largest G
//   w_j = scale * s_(e_j), divided by the sum of the chosen s with MOE_RENORM
//
// A masked expert (logit -inf or NaN) has s = 0 and ranks behind every other
// expert of the kept groups.  Scores, choices and group scores are held in
// fp64: two experts then rank as their exact scores do except within about
// 1e-15 of each other, and the choice does not depend on the order in which a
// softmax sum is formed.  An fp64 exp costs about 40 vector instructions,
// small beside the selection; measured with the rest below.
//
// One wave owns a token.  Lane l holds experts l*NV .. l*NV+NV-1 as 64-bit
// keys whose unsigned order is the order of the choices (0: not selectable,
// 1: masked), so a lower lane always holds lower indices.  Selection:
//  1. each lane's largest key is ranked among the 64 lanes by counting larger
//     ones; the k-th largest of them is a lower bound of the k-th largest key;
//  2. the keys not below that bound (k plus a few) are compacted, one per
//     lane, and ranked by counting; ranks below k are the answer, in order.
// More than 64 candidates (long ties, few lanes in the kept groups) take k
// rounds of a wave-wide maximum instead.
#include "k_sort_common.h"

namespace moe {

constexpr int RS_WAVES = 4;          // waves (tokens) per workgroup
constexpr int RSP_MAX_T = 16;        // one-workgroup select + sort up to this T
constexpr int RSP_MAX_KEYS = 8192;   // and up to this T*E: 64 KB of keys beside 34 KB of scratch

// Per-wave LDS of the selection.
struct SelScratch {
    uint64_t key[64];
    double score[64];
    uint64_t ckey[64];
    int cidx[64];
};

template <typename LT>
__device__ __forceinline__ float logit_f32(LT v);
template <>
__device__ __forceinline__ float logit_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float logit_f32<f16>(f16 v) { return (float)v; }
template <>
__device__ __forceinline__ float logit_f32<uint16_t>(uint16_t v)   // bf16 bits
{
    return __builtin_bit_cast(float, (uint32_t)v << 16);
}

// Monotonic key of a choice: larger choice, larger key; NaN counts as masked.
__device__ __forceinline__ uint64_t choice_key(double c, bool masked)
{
    if (masked || c != c)
        return 1ull;
    const int64_t b = __builtin_bit_cast(int64_t, c + 0.0);   // -0 ties with +0
    return (uint64_t)(b ^ ((b >> 63) | (int64_t)0x8000000000000000ull));
}

__device__ __forceinline__ double key_choice(uint64_t k)
{
    const int64_t b = (k >> 63) ? (int64_t)(k ^ 0x8000000000000000ull) : (int64_t)~k;
    return __builtin_bit_cast(double, b);
}

__device__ __forceinline__ double shfl_xor_f64(double v, int m)
{
    return __shfl_xor(v, m, 64);
}

__device__ __forceinline__ uint64_t readlane_u64(uint64_t v, int l)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l);
    return ((uint64_t)hi << 32) | lo;
}

struct SelArgs {
    const void *logits;
    int64_t ld;
    const float *bias;
    int T, E, k, score, n_group, keep;
    unsigned flags;
    float scale;
    int32_t *idx;
    float *w;
};

// Two largest of a multiset of choices, as keys (0: none).
struct Top2 {
    uint64_t a, b;
};
__device__ __forceinline__ void top2_add(Top2 &t, uint64_t k)
{
    const uint64_t lo = k < t.a ? k : t.a;
    t.a = k < t.a ? t.a : k;
    t.b = lo < t.b ? t.b : lo;
}

// A group's rank key from its two largest keys (masked keys do not count).
__device__ __forceinline__ uint64_t group_key(Top2 t, bool top2)
{
    if (t.a <= 1ull)
        return 1ull;
    if (!top2 || t.b <= 1ull)
        return t.a;
    return choice_key(key_choice(t.a) + key_choice(t.b), false);
}

// Selection of token t by one wave.  gk: LDS of E keys, only read when the
// groups do not fall on whole power-of-two runs of lanes.  sidx (LDS) also
// receives the chosen experts when given.
template <int NV, typename LT>
__device__ __forceinline__ void select_token(const SelArgs &a, int t, int lane, SelScratch *sc,
                                             uint64_t *gk, int *sidx)
{
    const LT *row = static_cast<const LT *>(a.logits) + (int64_t)t * a.ld;
    const int e0 = lane * NV;
    const int E = a.E, k = a.k;
    float l[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        l[i] = e0 + i < E ? logit_f32<LT>(row[e0 + i]) : -__builtin_inff();
    float b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        b[i] = (a.bias && e0 + i < E) ? a.bias[e0 + i] : 0.0f;

    // masked: -inf or NaN; +inf counts as the largest finite value
    bool live[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        live[i] = l[i] > -__builtin_inff();
        l[i] = fminf(l[i], 3.402823466e38f);
    }
    double s[NV];
    if (a.score == MOE_SCORE_SOFTMAX) {
        float m = -3.402823466e38f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            m = live[i] ? fmaxf(m, l[i]) : m;
#pragma unroll
        for (int o = 32; o; o >>= 1)
            m = fmaxf(m, __shfl_xor(m, o, 64));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            s[i] = live[i] ? exp((double)l[i] - (double)m) : 0.0;
            sum += s[i];
        }
#pragma unroll
        for (int o = 32; o; o >>= 1)
            sum += shfl_xor_f64(sum, o);
        const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            s[i] *= inv;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            s[i] = live[i] ? 1.0 / (1.0 + exp(-(double)l[i])) : 0.0;
    }
    uint64_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        key[i] = e0 + i < E ? choice_key(s[i] + (double)b[i], !live[i]) : 0ull;

    if (a.keep < a.n_group) {
        const int size = E / a.n_group;
        const int per = size / NV;   // lanes per group, if whole
        const bool top2 = (a.flags & MOE_GROUP_TOP2) != 0;
        uint64_t mine;               // lane g < n_group: group g's rank key
        if (size % NV == 0 && (per & (per - 1)) == 0) {
            Top2 p{0ull, 0ull};
#pragma unroll
            for (int i = 0; i < NV; ++i)
                top2_add(p, key[i]);
            for (int o = 1; o < per; o <<= 1) {
                const Top2 q{__shfl_xor(p.a, o, 64), __shfl_xor(p.b, o, 64)};
                top2_add(p, q.a);
                top2_add(p, q.b);
            }
            mine = __shfl(group_key(p, top2), min(lane * per, 63), 64);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (e0 + i < E)
                    gk[e0 + i] = key[i];
            wave_lds_sync();
            Top2 p{0ull, 0ull};
            if (lane < a.n_group)
                for (int i = 0; i < size; ++i)
                    top2_add(p, gk[lane * size + i]);
            mine = group_key(p, top2);
            wave_lds_sync();
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const uint64_t o = readlane_u64(mine, g);
            rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
        }
        const uint64_t kept = __ballot(lane < a.n_group && rank < a.keep);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = e0 + i;
            if (e < E && !((kept >> (e / size)) & 1ull))
                key[i] = 0ull;
        }
    }

    // 1. a bound from the lanes' largest keys
    uint64_t mk = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i)
        mk = key[i] > mk ? key[i] : mk;
    sc->key[lane] = mk;
    wave_lds_sync();
    int r0 = 0, r1 = 0;
#pragma unroll
    for (int j = 0; j < 64; j += 2) {
        const uint4_t q = *reinterpret_cast<const uint4_t *>(&sc->key[j]);
        const uint64_t ka = ((uint64_t)q.y << 32) | q.x, kb = ((uint64_t)q.w << 32) | q.z;
        r0 += (ka > mk || (ka == mk && j < lane)) ? 1 : 0;
        r1 += (kb > mk || (kb == mk && j + 1 < lane)) ? 1 : 0;
    }
    const int lrank = r0 + r1;
    const uint64_t at = __ballot(lrank == k - 1);   // exactly one lane
    uint64_t bound = readlane_u64(mk, __ffsll((long long)at) - 1);
    bound = bound ? bound : 1ull;

    // 2. candidates, compacted in index order within each register
    const uint64_t below = (lane == 0) ? 0ull : (~0ull >> (64 - lane));
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        n += __popcll(__ballot(key[i] >= bound));
    int rank = 64, e = 0;
    double sv = 0.0;
    if (n <= 64) {
        int base = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool c = key[i] >= bound;
            const uint64_t m = __ballot(c);
            if (c) {
                const int p = base + __popcll(m & below);
                sc->ckey[p] = key[i];
                sc->cidx[p] = e0 + i;
                sc->score[p] = s[i];
            }
            base += __popcll(m);
        }
        wave_lds_sync();
        if (lane < n) {
            const uint64_t me = sc->ckey[lane];
            e = sc->cidx[lane];
            sv = sc->score[lane];
            int r = 0;
            for (int j = 0; j < n; ++j) {
                const uint64_t o = sc->ckey[j];
                r += (o > me || (o == me && sc->cidx[j] < e)) ? 1 : 0;
            }
            rank = r;
        }
    } else {
        for (int j = 0; j < k; ++j) {
            uint64_t best = key[0];
#pragma unroll
            for (int i = 1; i < NV; ++i)
                best = key[i] > best ? key[i] : best;
            const uint64_t top = wave_max_u64(best);
            // lowest lane holding it, then its lowest register: lowest index
            const int from = __ffsll((long long)__ballot(best == top)) - 1;
            int pick = -1;
            double ps = 0.0;
            if (lane == from) {
#pragma unroll
                for (int i = NV - 1; i >= 0; --i)
                    if (key[i] == top) {
                        pick = i;
                        ps = s[i];
                    }
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i == pick)
                        key[i] = 0ull;
            }
            const int pe = __shfl(e0 + pick, from, 64);
            const double pv = __shfl(ps, from, 64);
            if (lane == j) {
                rank = j;
                e = pe;
                sv = pv;
            }
        }
    }
    const bool sel = rank < k;
    double w = sel ? sv : 0.0;
    if (a.flags & MOE_RENORM) {
        double sum = w;
#pragma unroll
        for (int o = 32; o; o >>= 1)
            sum += shfl_xor_f64(sum, o);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (sel) {
        a.idx[(int64_t)t * k + rank] = e;
        a.w[(int64_t)t * k + rank] = (float)(w * (double)a.scale);
        if (sidx)
            sidx[rank] = e;
    }
    wave_lds_sync();   // the scratch may be reused for the wave's next token
}

// LDS of keys per wave for groups that do not fall on whole runs of lanes.
static size_t group_lds(const SelArgs &a, int NV)
{
    if (a.keep >= a.n_group)
        return 0;
    const int size = a.E / a.n_group, per = size / NV;
    const bool whole = size % NV == 0 && (per & (per - 1)) == 0;
    return whole ? 0 : (size_t)a.E * sizeof(uint64_t);
}

template <int NV, typename LT>
__global__ __launch_bounds__(RS_WAVES * 64) void route_select_kernel(SelArgs a)
{
    extern __shared__ __align__(16) uint64_t gkeys[];
    __shared__ __align__(16) SelScratch sc[RS_WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x * RS_WAVES + wave;
    if (t >= a.T)
        return;
    select_token<NV, LT>(a, t, lane, &sc[wave], gkeys + (size_t)wave * a.E, nullptr);
}

// At most RSP_MAX_T tokens: selection by one wave per token, then the stable
// sort of the T*k chosen experts by wave 0 -- one launch for a decode step.
template <int NV, typename LT>
__global__ __launch_bounds__(RSP_MAX_T * 64) void route_select_sort_kernel(
    SelArgs a, int32_t *__restrict__ counts, int32_t *__restrict__ offsets,
    int32_t *__restrict__ perm, int32_t *__restrict__ inv_perm)
{
    extern __shared__ __align__(16) uint64_t gkeys[];
    __shared__ __align__(16) SelScratch sc[RSP_MAX_T];
    __shared__ int sidx[RSP_MAX_T * 16];
    __shared__ int cnt[1024];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (wave < a.T)
        select_token<NV, LT>(a, wave, lane, &sc[wave], gkeys + (size_t)wave * a.E,
                             sidx + wave * a.k);
    lds_barrier();
    if (wave == 0) {
        const int n = a.T * a.k;
        wave_count_scan(sidx, n, a.E, cnt, counts, offsets, lane);
        wave_stable_positions(sidx, n, perm, inv_perm, lane);
    }
}

template <typename LT, typename F>
static int for_width(int E, F &&f)
{
    const int nv = (E + 63) / 64;
    if (nv <= 1) return f(std::integral_constant<int, 1>());
    if (nv <= 2) return f(std::integral_constant<int, 2>());
    if (nv <= 4) return f(std::integral_constant<int, 4>());
    if (nv <= 8) return f(std::integral_constant<int, 8>());
    return f(std::integral_constant<int, 16>());
}

template <typename LT>
static int launch_select_t(const SelArgs &a, int32_t *counts, int32_t *offsets, int32_t *perm,
                           int32_t *inv_perm, hipStream_t st)
{
    return for_width<LT>(a.E, [&](auto nv) -> int {
        constexpr int NV = decltype(nv)::value;
        const size_t g = group_lds(a, NV);
        if (counts) {
            static bool attr_set = false;   // raising the LDS limit is idempotent
            if (g && !attr_set) {
                MOE_HIP_TRY(hipFuncSetAttribute(
                    (const void *)route_select_sort_kernel<NV, LT>,
                    hipFuncAttributeMaxDynamicSharedMemorySize, RSP_MAX_KEYS * 8));
                attr_set = true;
            }
            hipLaunchKernelGGL((route_select_sort_kernel<NV, LT>), dim3(1), dim3(a.T * 64),
                               g * a.T, st, a, counts, offsets, perm, inv_perm);
            MOE_LAUNCH_CHECK("route_select_sort_kernel");
            return MOE_OK;
        }
        hipLaunchKernelGGL((route_select_kernel<NV, LT>), dim3((a.T + RS_WAVES - 1) / RS_WAVES),
                           dim3(RS_WAVES * 64), g * RS_WAVES, st, a);
        MOE_LAUNCH_CHECK("route_select_kernel");
        return MOE_OK;
    });
}

bool route_select_sorts(int T, int E)
{
    return T > 0 && T <= RSP_MAX_T && T * E <= RSP_MAX_KEYS;
}

// counts != NULL (route_select_sorts): with the sort, in one launch.
int launch_route_select(const void *logits, int dtype, int64_t ld, const float *bias, int T, int E,
                        int k, int score, int n_group, int keep, unsigned flags, float scale,
                        int32_t *idx, float *w, int32_t *counts, int32_t *offsets, int32_t *perm,
                        int32_t *inv_perm, hipStream_t st)
{
    const SelArgs a{logits, ld, bias, T, E, k, score, n_group, keep, flags, scale, idx, w};
    if (dtype == MOE_DTYPE_F32)
        return launch_select_t<float>(a, counts, offsets, perm, inv_perm, st);
    if (dtype == MOE_DTYPE_F16)
        return launch_select_t<f16>(a, counts, offsets, perm, inv_perm, st);
    return launch_select_t<uint16_t>(a, counts, offsets, perm, inv_perm, st);
}

// Router logits of at most 8 tokens, one wave per expert: the summation order
// of every other router kernel (partial j in lane j, then the xor butterfly),
// so the same bits.
template <int H, int TT>
__global__ __launch_bounds__(256) void route_logits_rows_kernel(
    const f16 *__restrict__ x, const f16 *__restrict__ wr, const float *__restrict__ bias, int T,
    int E, float *__restrict__ logits)
{
    constexpr int NCH = H / 8;
    constexpr int NCL = (NCH + 63) / 64;
    const int lane = threadIdx.x & 63;
    const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (e >= E)
        return;
    half8_t wv[NCL], xv[NCL][TT];
#pragma unroll
    for (int m = 0; m < NCL; ++m) {
        const int c = min(lane + 64 * m, NCH - 1);
        wv[m] = *reinterpret_cast<const half8_t *>(wr + (size_t)e * H + c * 8);
#pragma unroll
        for (int t = 0; t < TT; ++t)
            xv[m][t] = *reinterpret_cast<const half8_t *>(x + (size_t)min(t, T - 1) * H + c * 8);
    }
    const float b = bias ? bias[e] : 0.0f;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        float acc = 0.0f;
#pragma unroll
        for (int m = 0; m < NCL; ++m)
            if (lane + 64 * m < NCH) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc = __builtin_fmaf((float)xv[m][t][i], (float)wv[m][i], acc);
            }
        float v = pinned_xor_sum(acc, lane);
        if (bias)
            v = v + b;
        if (lane == 0 && t < T)
            logits[(size_t)t * E + e] = v;
    }
}

template <int H>
static int launch_logits_h(const f16 *x, const f16 *wr, const float *bias, int T, int E,
                           float *logits, hipStream_t s)
{
    const dim3 grid((E + 3) / 4), block(256);
    if (T <= 1)
        hipLaunchKernelGGL((route_logits_rows_kernel<H, 1>), grid, block, 0, s, x, wr, bias, T, E,
                           logits);
    else if (T <= 2)
        hipLaunchKernelGGL((route_logits_rows_kernel<H, 2>), grid, block, 0, s, x, wr, bias, T, E,
                           logits);
    else
        hipLaunchKernelGGL((route_logits_rows_kernel<H, 4>), grid, block, 0, s, x, wr, bias, T, E,
                           logits);
    MOE_LAUNCH_CHECK("route_logits_rows_kernel");
    return MOE_OK;
}

// T <= 4
int launch_route_logits_rows(const void *x, const void *wr, const float *bias, int T, int H, int E,
                             float *logits, hipStream_t s)
{
    const f16 *xh = static_cast<const f16 *>(x), *wh = static_cast<const f16 *>(wr);
    switch (H) {
    case 256: return launch_logits_h<256>(xh, wh, bias, T, E, logits, s);
    case 512: return launch_logits_h<512>(xh, wh, bias, T, E, logits, s);
    case 1024: return launch_logits_h<1024>(xh, wh, bias, T, E, logits, s);
    case 2048: return launch_logits_h<2048>(xh, wh, bias, T, E, logits, s);
    default: return set_error(MOE_EUNSUPPORTED, "router logits: H=%d not instantiated", H);
    }
}

}  // namespace moe
