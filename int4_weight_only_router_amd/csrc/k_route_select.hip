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
// softmax sum is formed.  exp and the reciprocal are written out for the range
// that occurs (20 and 6 fp64 instructions, at the full vector rate).
//
// One wave owns a token.  Lane l holds experts l*NV .. l*NV+NV-1 as 64-bit
// keys whose unsigned order is the order of the choices (0: not selectable,
// 1: masked), so a lower lane always holds lower indices.  Selection:
//  1. the lanes' largest keys, cut to their high words, are ranked among the
//     64 lanes by counting larger ones; the k-th largest is a lower bound of
//     the k-th largest key;
//  2. the keys not below that bound (k plus a few) are compacted, one per
//     lane, and ranked in full by counting; ranks below k are the answer, in
//     order.
// More than 64 candidates (long ties, few lanes in the kept groups) take k
// rounds of a wave-wide maximum instead.
//
// The grouping by expert follows in the same launch for a few tokens.  For
// more, a workgroup selects for 16 tokens and leaves how often it chose each
// expert; in a second launch each workgroup adds up what the others left (its
// own start in every expert's run) and places its elements: no order depends on
// timing.
//
// Measured: 1 x 64 2.8 us; 777 x 60 top-4 in 6 groups 6.8 + 4.3; 4096 x 512
// top-10 in 8 groups 13.4 + 6.7 (8.4 MB of logits are 1.6 us of that).  Of the 49 k
// cycles of the last's selection a SIMD issues vector instructions in 17 k (1070
// a token, a third of them fp64), and waves wait 54% of theirs: steps through
// LDS and across lanes that depend on each other.  Placement reads every chunk's
// counts in every workgroup (33 MB from the L2) and scatters with one wave.
#include "k_sort_common.h"

namespace moe {

constexpr int RS_WAVES = 4;          // waves (tokens) per workgroup
constexpr int RSP_MAX_T = 16;        // one-workgroup select + sort up to this T
constexpr int RSP_MAX_KEYS = 8192;   // and up to this T*E: 64 KB of keys beside 34 KB of scratch
constexpr int RSC_WAVES = 16;        // chunked form: waves per workgroup,
constexpr int RSC_TOK = 16;          // tokens of a chunk,
constexpr int RSC_MAX_T = 8192;      // tokens up to which it is used,
constexpr size_t RSC_KEY_BYTES = 96 * 1024;   // LDS for group keys beside its scratch

size_t permute_ws_bytes(int T, int k, int E);
int launch_permute(const int32_t *, int, int, int, int32_t *, int32_t *, int32_t *, int32_t *,
                   void *, hipStream_t);

// Per-wave LDS of the selection.
struct SelScratch {
    uint32_t key[64];
    double score[64];
    uint64_t ckey[64 + 4];   // and four zeros behind the last candidate
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

// exp(x) for x <= 709 (0 below -745): x = n ln 2 + r, |r| about ln 2 / 2 at
// most, Taylor to r^13 (next term 4e-18).  The reduction is Cody and Waite's
// (Software Manual for the Elementary Functions, 1980), ln 2 in two parts; with
// fma the first may be ln 2 rounded to fp64 itself, LN2 = 0x1.62e42fefa39efp-1:
// it is a multiple of 2^-53, x one of 2^-53 (|x| >= 1/2) or of 2^-54 (|x| >= 1/4,
// then |n| <= 1, and below that n = 0), so x - n LN2, smaller than 1/2, fits 53
// bits and is exact.  LN2_LO = ln 2 - LN2, rounded.
__device__ __forceinline__ double exp_f64(double x)
{
    constexpr double LN2 = 0x1.62e42fefa39efp-1, LN2_LO = 0x1.abc9e3b39803fp-56;
    x = fmax(x, -746.0);
    const double n = __builtin_rint(x * (1.0 / LN2));
    double r = __builtin_fma(n, -LN2, x);
    r = __builtin_fma(n, -LN2_LO, r);
    double p = 1.0 / 6227020800.0;
    p = __builtin_fma(p, r, 1.0 / 479001600.0);
    p = __builtin_fma(p, r, 1.0 / 39916800.0);
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
    p = __builtin_fma(p, r, 1.0 / 362880.0);
    p = __builtin_fma(p, r, 1.0 / 40320.0);
    p = __builtin_fma(p, r, 1.0 / 5040.0);
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1 / x for 1 <= x < 2^1000: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double rcp_f64(double x)
{
    double y = __builtin_amdgcn_rcp(x);
    y = __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
    return __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
}

// Wave-wide fp64 sum and fp32 maximum in a fixed order, without LDS: steps
// inside the 16-lane rows, then the four rows by reading their lanes.
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double a)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, a);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double readlane_f64(double a, int l)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, a);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_sum_f64(double a)
{
    a += dpp_f64<0xB1>(a);
    a += dpp_f64<0x4E>(a);
    a += dpp_f64<0x141>(a);
    a += dpp_f64<0x140>(a);
    return (readlane_f64(a, 0) + readlane_f64(a, 16)) + (readlane_f64(a, 32) + readlane_f64(a, 48));
}
__device__ __forceinline__ float wave_max_f32(float a)
{
#define MOE_MAX_STEP(C)                                                                       \
    a = fmaxf(a, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(                       \
                     0, __builtin_bit_cast(int, a), C, 0xF, 0xF, false)))
    MOE_MAX_STEP(0xB1);
    MOE_MAX_STEP(0x4E);
    MOE_MAX_STEP(0x141);
    MOE_MAX_STEP(0x140);
#undef MOE_MAX_STEP
    float m = a;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        m = fmaxf(m, __builtin_bit_cast(
                         float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, a), 16 * r)));
    return m;
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

// What one token's selection left for its grouping: lane's rank (>= k: none).
struct SelOut {
    int rank, e;
};

// Selection of token t by one wave.  gk: LDS of E keys, only read when the
// groups do not fall on whole power-of-two runs of lanes.  sidx (LDS) also
// receives the chosen experts when given.
template <int NV, typename LT>
__device__ __forceinline__ SelOut select_token(const SelArgs &a, int t, int lane, SelScratch *sc,
                                             uint64_t *gk, int *sidx)
{
    const LT *row = static_cast<const LT *>(a.logits) + (int64_t)t * a.ld;
    const int e0 = lane * NV;
    const int E = a.E, k = a.k;
    float l[NV], b[NV];
    // a full row of 64 NV experts in 16-byte loads where it is aligned, else
    // one by one (past the end the last expert's, then masked: nothing is
    // predicated)
    constexpr int VW = 16 / (int)sizeof(LT);
    if (NV % VW == 0 && E == 64 * NV && ((uintptr_t)row & 15) == 0) {
        typedef LT lvec __attribute__((ext_vector_type(VW)));
#pragma unroll
        for (int i = 0; i < NV / VW; ++i) {
            const lvec v = *reinterpret_cast<const lvec *>(row + e0 + i * VW);
#pragma unroll
            for (int j = 0; j < VW; ++j)
                l[(i * VW + j) % NV] = logit_f32<LT>(v[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            l[i] = logit_f32<LT>(row[min(e0 + i, E - 1)]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            l[i] = e0 + i < E ? l[i] : -__builtin_inff();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        b[i] = 0.0f;
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            b[i] = a.bias[min(e0 + i, E - 1)];
    }

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
        m = wave_max_f32(m);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            s[i] = live[i] ? exp_f64((double)l[i] - (double)m) : 0.0;
            sum += s[i];
        }
        sum = wave_sum_f64(sum);
        const double inv = sum > 0.0 ? rcp_f64(sum) : 0.0;   // sum is 0 or at least 1
#pragma unroll
        for (int i = 0; i < NV; ++i)
            s[i] *= inv;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // with t = exp(-|l|) <= 1 nothing overflows at either end
            const double t = exp_f64(-fabs((double)l[i])), r = rcp_f64(1.0 + t);
            s[i] = !live[i] ? 0.0 : l[i] < 0.0f ? t * r : r;
        }
    }
    uint64_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        key[i] = e0 + i < E ? choice_key(s[i] + (double)b[i], !live[i]) : 0ull;

    if (a.keep < a.n_group) {
        const int size = E / a.n_group;
        const int per = size / NV;   // lanes per group, if whole
        const bool top2 = (a.flags & MOE_GROUP_TOP2) != 0;
        const bool whole = size % NV == 0 && (per & (per - 1)) == 0;
        uint64_t mine;               // lane g < n_group: group g's rank key
        if (whole) {
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
        if (whole) {   // a lane's experts are of one group
            const bool in = (kept >> min(e0 / size, 63)) & 1ull;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                key[i] = in ? key[i] : 0ull;
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = e0 + i;
                if (e < E && !((kept >> (e / size)) & 1ull))
                    key[i] = 0ull;
            }
        }
    }

    // 1. a bound from the lanes' largest keys: their high words, made unique
    // (and cut a little lower) by the lane
    uint64_t mk = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i)
        mk = key[i] > mk ? key[i] : mk;
    const uint32_t mine32 = ((uint32_t)(mk >> 32) & ~63u) | (uint32_t)(63 - lane);
    sc->key[lane] = mine32;
    wave_lds_sync();
    int r0 = 0, r1 = 0;
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
        const uint4_t v = *reinterpret_cast<const uint4_t *>(&sc->key[j]);
        r0 += v.x > mine32 ? 1 : 0;
        r1 += v.y > mine32 ? 1 : 0;
        r0 += v.z > mine32 ? 1 : 0;
        r1 += v.w > mine32 ? 1 : 0;
    }
    const uint64_t at = __ballot(r0 + r1 == k - 1);   // exactly one lane
    const uint32_t cut = (uint32_t)__builtin_amdgcn_readlane((int)mine32,
                                                             __ffsll((long long)at) - 1) & ~63u;
    const uint64_t bound = cut ? (uint64_t)cut << 32 : 1ull;

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
        if (lane < 4)
            sc->ckey[n + lane] = 0ull;
        wave_lds_sync();
        const uint64_t me = lane < n ? sc->ckey[lane] : ~0ull;
        e = sc->cidx[lane];
        sv = sc->score[lane];
        int above = 0, same = 0;
        for (int j = 0; j < n; j += 4) {
            const uint4_t u = *reinterpret_cast<const uint4_t *>(&sc->ckey[j]);
            const uint4_t v = *reinterpret_cast<const uint4_t *>(&sc->ckey[j + 2]);
            const uint64_t o[4] = {((uint64_t)u.y << 32) | u.x, ((uint64_t)u.w << 32) | u.z,
                                   ((uint64_t)v.y << 32) | v.x, ((uint64_t)v.w << 32) | v.z};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                above += o[i] > me ? 1 : 0;
                same += o[i] == me ? 1 : 0;
            }
        }
        if (__any(lane < n && same > 1)) {   // ties: the lower expert first
            for (int j = 0; j < n; ++j)
                above += sc->ckey[j] == me && sc->cidx[j] < e ? 1 : 0;
        }
        rank = lane < n ? above : 64;
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
        const double sum = wave_sum_f64(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (sel) {
        a.idx[(int64_t)t * k + rank] = e;
        a.w[(int64_t)t * k + rank] = (float)(w * (double)a.scale);
        if (sidx)
            sidx[rank] = e;
    }
    wave_lds_sync();   // the scratch may be reused for the wave's next token
    return SelOut{sel ? rank : k, e};
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

// One token: its experts' places by marking them in LDS, without a sort.
template <int NV, typename LT>
__global__ __launch_bounds__(64) void route_select_one_kernel(
    SelArgs a, int32_t *__restrict__ counts, int32_t *__restrict__ offsets,
    int32_t *__restrict__ perm, int32_t *__restrict__ inv_perm)
{
    extern __shared__ __align__(16) uint64_t gkeys[];
    __shared__ __align__(16) SelScratch sc;
    __shared__ int mark[64 * NV];   // rank + 1 of a chosen expert
    const int lane = threadIdx.x;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        mark[lane * NV + i] = 0;
    const SelOut o = select_token<NV, LT>(a, 0, lane, &sc, gkeys, nullptr);
    if (o.rank < a.k)
        mark[o.e] = o.rank + 1;
    wave_lds_sync();
    int m[NV], n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        m[i] = mark[lane * NV + i];
        n += m[i] != 0;
    }
    int at = n;
#pragma unroll
    for (int st = 1; st < 64; st <<= 1) {
        const int v = __shfl_up(at, st, 64);
        if (lane >= st)
            at += v;
    }
    at -= n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        if (e < a.E) {
            counts[e] = m[i] != 0;
            offsets[e] = at;
        }
        if (m[i]) {
            perm[at] = m[i] - 1;
            inv_perm[m[i] - 1] = at;
            ++at;
        }
    }
    if (lane == 0)
        offsets[a.E] = a.k;
}

// Chunked form, first launch: selection of RSC_TOK tokens per workgroup and
// how often they chose each expert (at most once per token: a byte).
template <int NV, typename LT>
__global__ __launch_bounds__(RSC_WAVES * 64) void route_select_count_kernel(
    SelArgs a, uint8_t *__restrict__ hist)
{
    extern __shared__ __align__(16) uint64_t gkeys[];
    __shared__ __align__(16) SelScratch sc[RSC_WAVES];
    __shared__ int cnt[1024];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    cnt[threadIdx.x] = 0;
    lds_barrier();
    for (int i = 0; i < RSC_TOK / RSC_WAVES; ++i) {
        const int t = blockIdx.x * RSC_TOK + i * RSC_WAVES + wave;
        if (t < a.T) {
            const SelOut o = select_token<NV, LT>(a, t, lane, &sc[wave],
                                                  gkeys + (size_t)wave * a.E, nullptr);
            if (o.rank < a.k)
                atomicAdd(&cnt[o.e], 1);
        }
    }
    lds_barrier();
    const int pitch = (a.E + 15) & ~15;
    if ((int)threadIdx.x < pitch)   // cnt past E is zero
        hist[(size_t)blockIdx.x * pitch + threadIdx.x] = (uint8_t)cnt[threadIdx.x];
}

// Second launch: workgroup b places chunk b's elements.  Thread (g, e) adds up
// every G-th chunk's counts of experts 16e..16e+15, in all chunks and in those
// before b (16-bit lanes: at most 16 * RSC_MAX_T / RSC_TOK).
__global__ __launch_bounds__(1024) void route_place_kernel(
    const int32_t *__restrict__ idx, const uint4_t *__restrict__ hist, int T, int k, int E,
    int chunks, int32_t *__restrict__ counts, int32_t *__restrict__ offsets,
    int32_t *__restrict__ perm, int32_t *__restrict__ inv_perm)
{
    __shared__ int tot[1024], pre[1024], wsum[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int mine = blockIdx.x;
    tot[tid] = 0;
    pre[tid] = 0;
    lds_barrier();
    const int EV = (E + 15) / 16, G = 1024 / EV, g = tid / EV, e = tid - g * EV;
    if (g < G && g < chunks) {
        uint32_t all[8], bef[8];   // [2 w + h]: experts 4w + h and 4w + h + 2
#pragma unroll
        for (int i = 0; i < 8; ++i)
            all[i] = bef[i] = 0u;
        for (int b0 = g; b0 < chunks; b0 += 4 * G) {
            uint4_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = hist[(size_t)min(b0 + i * G, chunks - 1) * EV + e];
            // four chunks add up within their bytes (at most 16 each)
            uint4_t v4 = {0u, 0u, 0u, 0u}, u4 = v4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int b = b0 + i * G;
                const uint32_t in = b < chunks ? ~0u : 0u, before = b < mine ? ~0u : 0u;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    v4[w] += h[i][w] & in;
                    u4[w] += h[i][w] & before;
                }
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                all[2 * w] += v4[w] & 0x00ff00ffu;
                all[2 * w + 1] += (v4[w] >> 8) & 0x00ff00ffu;
                bef[2 * w] += u4[w] & 0x00ff00ffu;
                bef[2 * w + 1] += (u4[w] >> 8) & 0x00ff00ffu;
            }
        }
        // zeros are most of a chunk's counts: only the others meet in LDS
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = 16 * e + 4 * (i >> 1) + (i & 1);
            if (all[i] & 0xffffu)
                atomicAdd(&tot[at], (int)(all[i] & 0xffffu));
            if (all[i] >> 16)
                atomicAdd(&tot[at + 2], (int)(all[i] >> 16));
            if (bef[i] & 0xffffu)
                atomicAdd(&pre[at], (int)(bef[i] & 0xffffu));
            if (bef[i] >> 16)
                atomicAdd(&pre[at + 2], (int)(bef[i] >> 16));
        }
    }
    lds_barrier();
    const int c = tid < E ? tot[tid] : 0;
    int incl = c;
#pragma unroll
    for (int st = 1; st < 64; st <<= 1) {
        const int v = __shfl_up(incl, st, 64);
        if (lane >= st)
            incl += v;
    }
    if (lane == 63)
        wsum[wave] = incl;
    lds_barrier();
    int off = incl - c;
    for (int i = 0; i < wave; ++i)
        off += wsum[i];
    if (tid < E) {
        if (mine == 0) {
            counts[tid] = c;
            offsets[tid] = off;
        }
        pre[tid] += off;
    }
    if (mine == 0 && tid == E - 1)
        offsets[E] = off + c;
    lds_barrier();
    if (wave == 0) {
        const int f0 = mine * RSC_TOK * k, f1 = min(T * k, f0 + RSC_TOK * k);
        wave_scatter(idx, f0, f1, E, pre, perm, inv_perm, lane);
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

// The grouping's outputs (counts NULL: selection alone); hist: the chunked form.
struct SelSort {
    int32_t *counts, *offsets, *perm, *inv_perm;
    uint8_t *hist;
};

template <typename LT>
static int launch_select_t(const SelArgs &a, const SelSort &how, hipStream_t st)
{
    return for_width<LT>(a.E, [&](auto nv) -> int {
        constexpr int NV = decltype(nv)::value;
        const size_t g = group_lds(a, NV);
        if (how.counts && a.T == 1) {
            hipLaunchKernelGGL((route_select_one_kernel<NV, LT>), dim3(1), dim3(64), g, st, a,
                               how.counts, how.offsets, how.perm, how.inv_perm);
            MOE_LAUNCH_CHECK("route_select_one_kernel");
            return MOE_OK;
        }
        if (how.counts && how.hist) {
            static LdsLimit limit;
            if (g)   // group keys
                if (const int rc = limit.raise((const void *)route_select_count_kernel<NV, LT>,
                                               (int)RSC_KEY_BYTES))
                    return rc;
            const int chunks = (a.T + RSC_TOK - 1) / RSC_TOK;
            hipLaunchKernelGGL((route_select_count_kernel<NV, LT>), dim3(chunks),
                               dim3(RSC_WAVES * 64), g * RSC_WAVES, st, a, how.hist);
            MOE_LAUNCH_CHECK("route_select_count_kernel");
            hipLaunchKernelGGL(route_place_kernel, dim3(chunks), dim3(1024), 0, st, a.idx,
                               reinterpret_cast<const uint4_t *>(how.hist),
                               a.T, a.k, a.E, chunks, how.counts, how.offsets, how.perm,
                               how.inv_perm);
            MOE_LAUNCH_CHECK("route_place_kernel");
            return MOE_OK;
        }
        if (how.counts) {
            static LdsLimit limit;
            if (g)   // group keys
                if (const int rc = limit.raise((const void *)route_select_sort_kernel<NV, LT>,
                                               (int)RSC_KEY_BYTES))
                    return rc;
            hipLaunchKernelGGL((route_select_sort_kernel<NV, LT>), dim3(1), dim3(a.T * 64),
                               g * a.T, st, a, how.counts, how.offsets, how.perm, how.inv_perm);
            MOE_LAUNCH_CHECK("route_select_sort_kernel");
            return MOE_OK;
        }
        hipLaunchKernelGGL((route_select_kernel<NV, LT>), dim3((a.T + RS_WAVES - 1) / RS_WAVES),
                           dim3(RS_WAVES * 64), g * RS_WAVES, st, a);
        MOE_LAUNCH_CHECK("route_select_kernel");
        return MOE_OK;
    });
}

// How the grouping is formed: inside the selecting workgroup, in chunks over
// two launches, or by the permutation's own launches behind the selection.
// Measured at 4096 tokens of 512 experts, top-10: 2 launches against 4.
enum { SORT_INSIDE, SORT_CHUNKS, SORT_AFTER };
static int sort_kind(int T, int E)
{
    if (T <= RSP_MAX_T && (T == 1 || T * E <= RSP_MAX_KEYS))
        return SORT_INSIDE;
    // the chunked form's 16 waves must fit their group keys in LDS
    if (T <= RSC_MAX_T && (size_t)E * 8 * RSC_WAVES <= RSC_KEY_BYTES)
        return SORT_CHUNKS;
    return SORT_AFTER;
}

size_t route_select_ws_bytes(int T, int k, int E)
{
    switch (sort_kind(T, E)) {
    case SORT_INSIDE: return T > 0 ? 0 : permute_ws_bytes(T, k, E);
    case SORT_CHUNKS: return (size_t)al256((int64_t)((T + RSC_TOK - 1) / RSC_TOK) * ((E + 15) & ~15));
    default: return permute_ws_bytes(T, k, E);
    }
}

// counts NULL: selection alone.
int launch_route_select(const void *logits, int dtype, int64_t ld, const float *bias, int T, int E,
                        int k, int score, int n_group, int keep, unsigned flags, float scale,
                        int32_t *idx, float *w, int32_t *counts, int32_t *offsets, int32_t *perm,
                        int32_t *inv_perm, void *ws, hipStream_t st)
{
    const SelArgs a{logits, ld, bias, T, E, k, score, n_group, keep, flags, scale, idx, w};
    const int kind = sort_kind(T, E);
    SelSort how{counts, offsets, perm, inv_perm, nullptr};
    if (counts && kind == SORT_CHUNKS)
        how.hist = static_cast<uint8_t *>(ws);
    if (kind == SORT_AFTER)
        how.counts = nullptr;
    if (T > 0) {
        const int rc = dtype == MOE_DTYPE_F32   ? launch_select_t<float>(a, how, st)
                       : dtype == MOE_DTYPE_F16 ? launch_select_t<f16>(a, how, st)
                                                : launch_select_t<uint16_t>(a, how, st);
        if (rc || !counts || kind != SORT_AFTER)
            return rc;
    }
    return counts ? launch_permute(idx, T, k, E, counts, offsets, perm, inv_perm, ws, st) : MOE_OK;
}

// Router logits of at most 4 tokens, one wave per expert: the summation order
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
