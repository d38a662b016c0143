// k_linear_tile.hip -- fp16 products of many rows on the matrix cores.
//
//   out[m][n] = residual + act(sum_k A(m, k) B(n, k) + bias[n])
//
// Tiles of BM x BN by WM x WN waves, each with its share of the tile in its
// accumulators; the small tiles by KG such groups of waves that share k and meet in
// LDS at the end.  Both operands travel to LDS by direct-to-LDS loads, 64 of k
// a stage, NS stages in flight.  An operand whose rows run along k lies in LDS as
// rows of 128 bytes, of which a lane reads the eight k of its matrix row; one
// whose rows run across k lies as 64 rows of BM (BN) values and is turned on the
// way to the registers by the transposing LDS read (four k of sixteen columns for
// sixteen lanes).  The pieces of a row are permuted so that the lanes of a read
// hit distinct banks; direct-to-LDS loads take consecutive lanes to consecutive
// 16-byte places, so the permutation is that of the lanes' source addresses.
//
// A stage is two steps of 32 of k.  A step's fragments are read during the step
// before it; the stage is changed in the middle of a block, when all its fragments
// are in registers: one barrier a block, behind which the stage takes the loads of
// the block NS later and the next block's first fragments are read.
//
// Bound by the matrix pipe where the tiles fill the card (4096 x 11264 x 2048: 174 us,
// 1.09 PFLOP/s, the pipe at work half of the cycles and the clock down to 2 GHz; the
// library's product 166 to 174), by the first loads and the results where they are a single
// round (333 x 1408 x 2000: 11 us), by bytes where K is short (4096 x 2048 x 64 to fp32:
// 10.8 us, 3.1 TB/s).
#include <algorithm>

#include "k_linear.h"

namespace moe {

typedef short short4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4_t lds_short4;

// The transposing read: of 16 lanes that give the addresses of four rows of sixteen
// values (four lanes a row, four values each), lane i gets column i.  (Without a
// restrict pointer the compiler takes the read to alias the direct-to-LDS loads in
// flight and waits for them; that they have arrived is shown by wait_vm and the
// barrier before it.)
__device__ __forceinline__ short4_t lds_turned(lds_short4 *__restrict__ p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

constexpr int LT_BK = 64;

// A tile's form.
template <int BM_, int BN_, int WM_, int WN_, int KG_, int NS_>
struct LtForm {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KG = KG_, NS = NS_;
    static constexpr int NTH = 64 * WM * WN;                     // threads of a group
    static constexpr int THREADS = NTH * KG;
    static constexpr int FM = BM / 16 / WM, FN = BN / 16 / WN;   // fragments of a wave
    static constexpr int STAGE = (BM + BN) * LT_BK * 2;          // bytes of a stage
    // The sums pass through LDS on their way out, in PASS parts of HR rows for each row
    // of waves; bytes of a row there, off the banks' period.
    static constexpr int ROW = BN * 4 + 16;
    static constexpr int PASS = KG * BM * ROW > 160 * 1024 ? 2 : 1, HR = BM / WM / PASS;
    static constexpr int ROW16 = BN * 2 + 16;   // the same, of fp16 results
    static constexpr int lds()
    {
        return std::max({KG * NS * STAGE, KG * BM / PASS * ROW, KG == 1 ? BM * ROW16 : 0});
    }
    static_assert(FM > 0 && FN > 0 && lds() <= 160 * 1024, "a tile's fragments and LDS");
};

// Which of its k an operand that runs across k gives: as they come; all of them twice
// over, starting again at `wrap`; or each of them twice in a row.
enum LtAgain { ONCE, OVER, EACH };

// One operand of a workgroup of NTH threads: R rows (of A or B) from row r0 on.
// AGAIN: not ONCE: k counts from k0 on, before the base.
template <int R, bool KS, int NTH, LtAgain AGAIN = ONCE>
struct LtOperand {
    static constexpr int LOADS = R * LT_BK * 2 / (NTH * 16);   // 16-byte loads a thread and block
    static constexpr int RB = KS ? R * 2 : LT_BK * 2;          // bytes of an LDS row
    static constexpr int PIECES = RB / 16;
    // Where a load of all threads fills whole LDS rows, their places repeat from load
    // to load LROWS rows on; else (24 pieces, 512 threads) every load has its own.
    static constexpr bool EVEN = NTH % PIECES == 0;
    static constexpr int LROWS = EVEN ? NTH / PIECES : 0, OWN = EVEN ? 1 : LOADS;
    const unsigned char *base;
    uint32_t ld, last;    // bytes: of a row; kc: of the last row (R <= 256, ld <= 2^24)
    int K, k0, wrap;
    uint32_t off[OWN];    // of this thread's (first) row
    uint32_t col[KS ? OWN : 1];   // ks: of its column

    static __device__ __forceinline__ int tid() { return (int)threadIdx.x % NTH; }
    // LDS row and piece of this thread's load i (EVEN: of the first one)
    static __device__ __forceinline__ int lrow(int i) { return (i * NTH + tid()) / PIECES; }
    static __device__ __forceinline__ int piece(int i)
    {
        return (i * NTH + tid()) % PIECES ^ turn(lrow(i));
    }
    // permutation of an LDS row's pieces
    static __device__ __forceinline__ int turn(int lrow)
    {
        if constexpr (!KS)
            return (lrow >> 1) & 7;
        else if constexpr (PIECES % 16 == 0)
            return ((lrow & 3) | ((lrow >> 3) & 1) << 2) * 2;
        else if constexpr (PIECES % 8 == 0)   // two rows a bank period, or one and a half
            return (((lrow >> 1) & 1) | ((lrow >> 3) & 1) << 1) * 2;
        else if constexpr (PIECES == 4)       // four
            return ((lrow >> 3) & 1) * 2;
        else
            return 0;
    }
    static_assert(LROWS % 16 == 0, "the permutation's period");
    // rows r0 .. rows - 1 of the operand, K of k
    __device__ __forceinline__ void init(const f16 *p, int64_t ld_, int r0, int rows, int K_)
    {
        ld = (uint32_t)ld_ * 2;
        K = K_;
        base = reinterpret_cast<const unsigned char *>(p + (KS ? (int64_t)r0 : (int64_t)r0 * ld_));
        last = (uint32_t)min(rows - r0 - 1, R - 1) * ld;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            off[i] = (uint32_t)lrow(i) * ld;
            if constexpr (KS)
                col[i] = (uint32_t)min(piece(i) * 8, ((rows - r0 + 7) & ~7) - 8) * 2;
        }
    }
    // load i of block kb to its place in the stage at `st`; rows and k past the end
    // read what lies at the end (a row is readable up to the next multiple of 8)
    __device__ __forceinline__ void load(int kb, int i, unsigned char *st) const
    {
        unsigned char *to = st + i * NTH * 16 + (tid() >> 6) * 1024;
        const uint32_t row = EVEN ? off[0] + (uint32_t)(i * LROWS) * ld : off[EVEN ? 0 : i];
        if constexpr (!KS) {
            const uint32_t k = min(kb * LT_BK + piece(0) * 8, ((K + 7) & ~7) - 8) * 2;
            dma16(base + (min(row, last) + k), to);
        } else {
            if constexpr (AGAIN != ONCE) {
                const int k = k0 + min(kb * LT_BK + lrow(i), K - 1);
                const int of = AGAIN == EACH ? k >> 1 : k < wrap ? k : k - wrap;
                dma16(base + (int64_t)of * ld + col[EVEN ? 0 : i], to);
                return;
            }
            const uint32_t end = (uint32_t)min(K - 1 - kb * LT_BK, LT_BK - 1) * ld;
            dma16(base + (int64_t)kb * LT_BK * ld + (min(row, end) + col[EVEN ? 0 : i]), to);
        }
    }
    // zeros where the stage of block kb holds no k of the product
    __device__ __forceinline__ void clear(int kb, unsigned char *st) const
    {
        const int k1 = K - kb * LT_BK;   // k of the block that exist
        const uint4_t z = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (KS ? lrow(i) >= k1 : piece(i) * 8 >= k1)
                *reinterpret_cast<uint4_t *>(st + (i * NTH + tid()) * 16) = z;
    }
    // fragment of the 16 rows from r (a multiple of 16) on, step s of a block
    static __device__ __forceinline__ half8_t frag(const unsigned char *st, int r, int s)
    {
        const int lane = threadIdx.x & 63;
        if constexpr (!KS) {
            return *reinterpret_cast<const half8_t *>(
                st + (r + (lane & 15)) * RB + ((s * 4 + (lane >> 4)) ^ turn(lane & 15)) * 16);
        } else {
            const int k = s * 32 + (lane >> 4) * 8 + ((lane & 15) >> 2);
            const int piece = (r >> 3) + ((lane & 3) >> 1);
            const unsigned char *at = st + k * RB + (piece ^ turn(k)) * 16 + (lane & 1) * 8;
            const short4_t a = lds_turned((lds_short4 *)at);
            const short4_t b = lds_turned((lds_short4 *)(at + 4 * RB));
            typedef short short8_t __attribute__((ext_vector_type(8)));
            const short8_t j = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(half8_t, j);
        }
    }
};

// The work item of a workgroup.  Workgroup i runs on XCD i % 8; each XCD takes a
// contiguous run of items, LT_GROUP row tiles before the next column tile, so that
// the tiles in flight on an XCD (32 compute units) share rows and weights in its L2.
constexpr int LT_NXCD = 8, LT_GROUP = 4;
struct LtItem {
    int mt, nt, split;
};
__device__ __forceinline__ bool lt_item(const LinArgs &a, int MT, int NT, LtItem &it)
{
    const int total = MT * NT * a.splits;
    const int run = (total + LT_NXCD - 1) / LT_NXCD;
    const int li = blockIdx.x / LT_NXCD;
    const int item = (int)(blockIdx.x % LT_NXCD) * run + li;
    if (li >= run || item >= total)
        return false;
    it.split = item / (MT * NT);
    const int tile = item - it.split * MT * NT;
    const int g = tile / (LT_GROUP * NT), r = tile - g * LT_GROUP * NT;
    const int gm = min(LT_GROUP, MT - g * LT_GROUP);
    it.mt = g * LT_GROUP + r % gm;
    it.nt = r / gm;
    return true;
}

template <typename F>
using LtAcc = float4_t[F::FM][F::FN];

// Columns n .. n + C - 1 of row m with the whole epilogue (v: their sums).
template <typename T, int C>
__device__ __forceinline__ void lt_finish(const LinArgs &a, T *out, int64_t m, int n, float (&v)[C],
                                          bool vec)
{
    const int cols = a.N - n;
    if (a.bias) {
        float b[C];
        load_piece<float, C>(a.bias + n, 0, cols, (uintptr_t)a.bias % 16 == 0, b);
#pragma unroll
        for (int j = 0; j < C; ++j)
            v[j] += b[j];
    }
    if (a.z)
        store_piece<f16, C>(a.z + m * a.ldz + n, 0, cols, vec, v);
    if (a.act != MOE_ACT_NONE)
#pragma unroll
        for (int j = 0; j < C; ++j)
            v[j] = act_value(v[j], a.act);
    if (a.residual) {
        float r[C];
        load_piece<T, C>(static_cast<const T *>(a.residual) + m * a.ldr + n, 0, cols, vec, r);
#pragma unroll
        for (int j = 0; j < C; ++j)
            v[j] += r[j];
    }
    store_piece<T, C>(out + m * a.ldo + n, 0, cols, vec, v);
}

// Whether every tensor of the epilogue can be read and written 16 bytes at a time.
template <typename T>
__device__ __forceinline__ bool lt_vec(const LinArgs &a, const T *out)
{
    auto rows16 = [](const void *p, int64_t ld, int size) {
        return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0;
    };
    return rows16(out, a.ldo, sizeof(T)) && (!a.residual || rows16(a.residual, a.ldr, sizeof(T))) &&
           (!a.z || rows16(a.z, a.ldz, 2));
}

// The sums through LDS, where the groups' meet in their order, and out in whole lines,
// C columns a thread: as many as keep the workgroup's threads at work.
template <typename F, typename T>
__device__ __forceinline__ void lt_epilogue(const LinArgs &a, LtAcc<F> &acc, const LtItem &it,
                                            int m0, int n0, int wm, int nw, unsigned char *smem)
{
    constexpr int LROWS = F::BM / F::PASS, MH = F::FM / F::PASS;
    constexpr int C = std::min(8, std::max(2, LROWS * F::BN / F::THREADS)), NP = F::BN / C;
    const int lane = threadIdx.x & 63, grp = threadIdx.x / F::NTH;
    T *out = static_cast<T *>(a.out) + it.split * a.split_stride;
    const bool vec = lt_vec<T>(a, out);
    auto at = [&](int g, int r, int c) {
        return reinterpret_cast<float *>(smem + (g * LROWS + r) * F::ROW + c * 4);
    };
#pragma unroll
    for (int h = 0; h < F::PASS; ++h) {
        __syncthreads();   // what was in LDS is read by all
#pragma unroll
        for (int m = 0; m < MH; ++m)
#pragma unroll
            for (int n = 0; n < F::FN; ++n)   // a lane holds four columns of a row
                *reinterpret_cast<float4_t *>(at(grp, wm * F::HR + m * 16 + (lane & 15),
                                                 nw + n * 16 + (lane >> 4) * 4)) = acc[h * MH + m][n];
        __syncthreads();
        for (int i = threadIdx.x; i < LROWS * NP; i += F::THREADS) {
            const int r = i / NP, c = i % NP * C;
            const int64_t m = m0 + r / F::HR * (F::BM / F::WM) + h * F::HR + r % F::HR;
            if (m >= a.M || n0 + c >= a.N)
                continue;
            float v[C];
            load_piece<float, C>(at(0, r, c), 0, C, true, v);
#pragma unroll
            for (int g = 1; g < F::KG; ++g) {
                float o[C];
                load_piece<float, C>(at(g, r, c), 0, C, true, o);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    v[j] += o[j];
            }
            lt_finish<T, C>(a, out, m, n0 + c, v, vec);
        }
    }
}

// The same where nothing but fp16 results leave: rounded before they pass through LDS,
// in one part (256 x 256, the same operands again and again: 4096 x 11264 x 2048 in 159
// us against 168).
template <typename F>
__device__ __forceinline__ void lt_epilogue_f16(const LinArgs &a, LtAcc<F> &acc, int m0, int n0,
                                                int mw, int nw, unsigned char *smem)
{
    constexpr int NP = F::BN / 8;
    const int lane = threadIdx.x & 63;
    f16 *out = static_cast<f16 *>(a.out);
    const bool vec = lt_vec<f16>(a, out);
    __syncthreads();   // the ring is read by all
#pragma unroll
    for (int n = 0; n < F::FN; ++n) {
        const int c = nw + n * 16 + (lane >> 4) * 4;
        float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (a.bias)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[j] = a.bias[min(n0 + c + j, a.N - 1)];
#pragma unroll
        for (int m = 0; m < F::FM; ++m) {
            half4_t v;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = (f16)(acc[m][n][j] + b[j]);
            *reinterpret_cast<half4_t *>(smem + (mw + m * 16 + (lane & 15)) * F::ROW16 + c * 2) = v;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < F::BM * NP; i += F::THREADS) {
        const int r = i / NP, c = i % NP * 8;
        const int64_t m = m0 + r;
        const int cols = a.N - (n0 + c);
        if (m >= a.M || cols <= 0)
            continue;
        const half8_t v = *reinterpret_cast<const half8_t *>(smem + r * F::ROW16 + c * 2);
        f16 *to = out + m * a.ldo + n0 + c;
        if (vec && cols >= 8) {
            *reinterpret_cast<half8_t *>(to) = v;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < cols)
                    to[j] = v[j];
        }
    }
}

// The same for fp32 results: straight from the registers, four columns of a row a lane,
// so that a store of the wave fills 64 bytes of each of 16 rows (128 x 128: 4096 x 2048 x
// 64 in 10.8 us, through LDS 12.3).
template <typename F>
__device__ __forceinline__ void lt_epilogue_f32(const LinArgs &a, LtAcc<F> &acc, float *out, int m0,
                                                int n0, int mw, int nw)
{
    const int lane = threadIdx.x & 63;
    const bool vec = (uintptr_t)out % 16 == 0 && a.ldo % 4 == 0;
#pragma unroll
    for (int n = 0; n < F::FN; ++n) {
        const int c = n0 + nw + n * 16 + (lane >> 4) * 4, cols = a.N - c;
        if (cols <= 0)
            continue;
        float4_t b = {0.0f, 0.0f, 0.0f, 0.0f};
        if (a.bias)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[j] = a.bias[min(c + j, a.N - 1)];
#pragma unroll
        for (int m = 0; m < F::FM; ++m) {
            const int64_t r = m0 + mw + m * 16 + (lane & 15);
            if (r >= a.M)
                continue;
            float *to = out + r * a.ldo + c;
            const float4_t v = acc[m][n] + b;
            if (vec && cols >= 4) {
                *reinterpret_cast<float4_t *>(to) = v;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < cols)
                        to[j] = v[j];
            }
        }
    }
}

template <typename F, bool AKS, bool BKS, LtAgain AGAIN>
__global__ __launch_bounds__(F::THREADS, 2) void linear_tile_kernel(LinArgs a)
{
    constexpr int BM = F::BM, BN = F::BN, NS = F::NS, STAGE = F::STAGE, FM = F::FM, FN = F::FN;
    typedef LtOperand<BM, AKS, F::NTH> OA;
    typedef LtOperand<BN, BKS, F::NTH, AGAIN> OB;
    constexpr int P = OA::LOADS + OB::LOADS;
    constexpr int AB = BM * LT_BK * 2;          // B's place in a stage
    // Of the row fragments the first ROLL are read into the registers that their own
    // sums have just left, the others into a second set: with two whole sets the
    // 256 x 256 tile is out of registers.
    constexpr int ROLL = FM > 4 ? FM / 2 : 0;
    extern __shared__ __align__(16) unsigned char smem[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % (F::WM * F::WN);
    const int grp = F::KG > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / F::NTH) : 0;
    const int mw = wave / F::WN * (BM / F::WM), nw = wave % F::WN * (BN / F::WN);

    LtItem it;
    if (!lt_item(a, (a.M + BM - 1) / BM, (a.N + BN - 1) / BN, it))
        return;
    const int m0 = it.mt * BM, n0 = it.nt * BN;
    // blocks of k: of this workgroup, of each group, of this one
    const int kall = (a.K + LT_BK - 1) / LT_BK, kw0 = it.split * a.kblocks;
    const int nw_kb = min(kall - kw0, a.kblocks);
    const int each = (nw_kb + F::KG - 1) / F::KG;
    const int kb0 = kw0 + grp * each;
    const int nkb = max(0, min(nw_kb - grp * each, each));
    const int K = min(a.K - min(kb0, kall - 1) * LT_BK, max(nkb, 1) * LT_BK);
    // the block with the end of k inside it, in the group that has it
    const int tail_grp = (nw_kb - 1) / each, tail_kb = nw_kb - 1 - tail_grp * each;
    const bool cut = kw0 + nw_kb == kall && a.K % LT_BK;
    unsigned char *ring = smem + grp * NS * STAGE;
    OA oa;
    OB ob;
    const int64_t k0 = (int64_t)min(kb0, kall - 1) * LT_BK;
    oa.init(a.a + k0 * (AKS ? a.lda : 1), a.lda, m0, a.M, K);
    ob.init(a.b + (AGAIN != ONCE ? 0 : k0 * (BKS ? a.ldb : 1)), a.ldb, n0, a.N, K);
    ob.k0 = (int)k0;
    ob.wrap = a.K / 2;

    LtAcc<F> acc;
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n)
            acc[m][n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

    auto load1 = [&](int kb, int i) {
        unsigned char *st = ring + kb % NS * STAGE;
        if (i < OA::LOADS)
            oa.load(kb, i, st);
        else
            ob.load(kb, i - OA::LOADS, st + AB);
    };
    half8_t fa[2][FM], fb[2][FN];
    auto read_a = [&](const unsigned char *st, int s, int m) {
        fa[m < ROLL ? 0 : s][m] = OA::frag(st, mw + m * 16, s);
    };
    auto read_b = [&](const unsigned char *st, int s, int n) {
        fb[s][n] = OB::frag(st + AB, nw + n * 16, s);
    };
    auto clear = [&](int kb) {   // behind the barrier that shows block kb
        if (cut && kb == tail_kb) {
            if (grp == tail_grp) {
                oa.clear(kb, ring + kb % NS * STAGE);
                ob.clear(kb, ring + kb % NS * STAGE + AB);
            }
            lds_barrier();
        }
    };
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (i < nkb)
#pragma unroll
            for (int j = 0; j < P; ++j)
                load1(i, j);
    if (nkb >= NS)
        wait_vm<(NS - 1) * P>();
    else
        wait_vm<0>();
    lds_barrier();
    clear(0);
#pragma unroll
    for (int i = 0; i < FN; ++i)
        read_b(ring, 0, i);
#pragma unroll
    for (int i = 0; i < FM; ++i)
        read_a(ring, 0, i);

    constexpr int T = FM * FN, R = FM + FN;   // sums and fragments of a step
    constexpr int RE = T / R > 0 ? T / R : 1;
    // read of the next step's fragment number i, in the order in which registers
    // come free: columns and rolling rows in turn, then the other rows
    auto read_next = [&](const unsigned char *st, int s, int i) {
        constexpr int LEAD = FN - ROLL / 2;   // columns before the first rolling row
        if (ROLL && i >= LEAD && i < LEAD + 2 * ROLL - 1) {
            const int j = i - LEAD;
            if (j % 2 == 0)
                read_a(st, s, j / 2);
            else if (LEAD + j / 2 < FN)
                read_b(st, s, LEAD + j / 2);
            else
                read_a(st, s, ROLL + j / 2 - (FN - LEAD));
        } else if (i < FN) {
            read_b(st, s, i);
        } else {
            read_a(st, s, i - FN);
        }
    };
    static_assert(!ROLL || (RE * (FN - ROLL / 2) >= FN && RE * 2 >= FN),
                  "a rolling row's registers are free when it is read");
    auto step = [&](int s, auto &&between) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const int m = i / FN, n = i % FN;
            between(i);

            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                fb[s][n], fa[m < ROLL ? 0 : s][m], acc[m][n], 0, 0, 0);
        }
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto block = [&](int kb, auto more) {
        constexpr bool MORE = decltype(more)::value;   // block kb + NS exists
        const unsigned char *st = ring + kb % NS * STAGE;
        step(0, [&](int i) {
            if (RE > 1 || R <= T) {
                if (i % RE == 0 && i / RE < R)
                    read_next(st, 1, i / RE);
            } else if (i == 0) {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    read_next(st, 1, j);
            }
        });
        if (MORE)
            wait_vm<(NS - 2) * P>();
        else
            wait_vm<0>();
        lds_barrier();
        if (!MORE || F::KG > 1)   // (groups may be at different numbers of blocks left)
            clear(kb + 1);
        const unsigned char *nx = ring + (kb + 1) % NS * STAGE;
        constexpr int PE = T / P > 0 ? T / P : 1;   // sums a load
        step(1, [&](int i) {
            if (RE > 1 || R <= T) {
                if (i % RE == 0 && i / RE < R)
                    read_next(nx, 0, i / RE);
            } else if (i == 0) {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    read_next(nx, 0, j);
            }
            if (MORE) {
                if (P <= T) {
                    if (i % PE == 0 && i / PE < P)
                        load1(kb + NS, i / PE);
                } else if (i == 0) {
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        load1(kb + NS, j);
                }
            }
        });
    };
    // every group passes as many barriers; one without a block's work adds nothing
    int kb = 0;
    for (; kb + NS < nkb; ++kb)
        block(kb, std::true_type());
    for (; kb < nkb; ++kb)
        block(kb, std::false_type());
    if constexpr (F::KG > 1)
        for (; kb < each; ++kb) {
            lds_barrier();
            clear(kb + 1);
        }
    if constexpr (F::KG == 1)
        if (a.act == MOE_ACT_NONE && !a.residual && !a.z) {
            if (a.odt == MOE_DTYPE_F16)
                lt_epilogue_f16<F>(a, acc, m0, n0, mw, nw, smem);
            else
                lt_epilogue_f32<F>(a, acc, static_cast<float *>(a.out) + it.split * a.split_stride,
                                   m0, n0, mw, nw);
            return;
        }
    if (a.odt == MOE_DTYPE_F32)
        lt_epilogue<F, float>(a, acc, it, m0, n0, wave / F::WN, nw, smem);
    else
        lt_epilogue<F, f16>(a, acc, it, m0, n0, wave / F::WN, nw, smem);
}

// Sums of the splits' partial products, in their order, with the epilogue; behind the
// `blocks` workgroups for them those of a.columns.
template <typename T>
__global__ __launch_bounds__(256) void linear_join_kernel(LinArgs a, const float *parts, int64_t ld,
                                                          int blocks)
{
    __shared__ float s[16][64];
    if ((int)blockIdx.x >= blocks) {
        column_sums<4>(a.columns, blockIdx.x - blocks, s);
        return;
    }
    const int64_t chunks = (a.N + 7) / 8, total = chunks * a.M;
    const bool vec = lt_vec<T>(a, static_cast<const T *>(a.out));
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < total; i += blocks * 256LL) {
        const int64_t m = i / chunks;
        const int n = (int)(i - m * chunks) * 8;
        const float *p = parts + m * ld + n;
        float v[8];
        load_piece<float, 8>(p, 0, 8, true, v);
        for (int s = 1; s < a.splits; ++s) {
            float w[8];
            load_piece<float, 8>(p + s * a.split_stride, 0, 8, true, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] += w[j];
        }
        lt_finish<T, 8>(a, static_cast<T *>(a.out), m, n, v, vec);
    }
}

template <typename F, bool AKS, bool BKS, LtAgain AGAIN>
static int launch_tile_t(const LinArgs &a, hipStream_t s)
{
    static LdsLimit limit;
    const int64_t items =
        (int64_t)((a.M + F::BM - 1) / F::BM) * ((a.N + F::BN - 1) / F::BN) * a.splits;
    const int rc = limit.raise((const void *)linear_tile_kernel<F, AKS, BKS, AGAIN>, 160 * 1024);
    if (rc)
        return rc;
    const unsigned grid = (unsigned)((items + LT_NXCD - 1) / LT_NXCD * LT_NXCD);
    hipLaunchKernelGGL((linear_tile_kernel<F, AKS, BKS, AGAIN>), dim3(grid), dim3(F::THREADS),
                       F::lds(), s, a);
    MOE_LAUNCH_CHECK("linear_tile_kernel");
    return MOE_OK;
}

// BOTH: the form takes products both of whose operands run across k (linear_plan chooses
// no other form for those).
template <typename F, bool BOTH>
static int launch_tile(const LinArgs &a, hipStream_t s)
{
    if (a.a_ks) {
        if constexpr (BOTH)
            return a.twice ? launch_tile_t<F, true, true, EACH>(a, s)
                           : launch_tile_t<F, true, true, ONCE>(a, s);
        return set_error(MOE_EUNSUPPORTED, "linear_tile_kernel: no such form");
    }
    if (a.b_ks)
        return a.twice ? launch_tile_t<F, false, true, OVER>(a, s)
                       : launch_tile_t<F, false, true, ONCE>(a, s);
    return launch_tile_t<F, false, false, ONCE>(a, s);
}

// The forms in the order of LinPlan::form (what each is for: linear_plan).
typedef LtForm<16, 32, 1, 2, 8, 3> LtF0;
typedef LtForm<32, 64, 1, 4, 2, 4> LtF1;
typedef LtForm<64, 64, 2, 2, 2, 4> LtF2;
typedef LtForm<64, 64, 2, 2, 1, 4> LtF3;
typedef LtForm<128, 128, 2, 4, 1, 4> LtF4;
typedef LtForm<128, 128, 2, 2, 1, 2> LtF5;
typedef LtForm<192, 256, 2, 4, 1, 2> LtF6;
typedef LtForm<256, 256, 2, 4, 1, 2> LtF7;
typedef LtForm<256, 128, 4, 2, 1, 3> LtF8;

int launch_linear_tile(LinArgs a, const LinPlan &p, void *ws, hipStream_t s)
{
    const int nkb = (a.K + LT_BK - 1) / LT_BK;
    a.kblocks = (nkb + p.splits - 1) / p.splits;
    a.splits = p.splits;
    LinArgs part = a;
    part.split_stride = 0;
    if (a.splits > 1) {
        const int64_t ld = (int64_t)(a.N + 7) / 8 * 8;
        part.bias = nullptr;
        part.act = MOE_ACT_NONE;
        part.residual = nullptr;
        part.z = nullptr;
        part.out = ws;
        part.odt = MOE_DTYPE_F32;
        part.ldo = ld;
        part.split_stride = ld * a.M;
    }
    int rc;
    switch (p.form) {
    case 0: rc = launch_tile<LtF0, false>(part, s); break;
    case 1: rc = launch_tile<LtF1, true>(part, s); break;
    case 2: rc = launch_tile<LtF2, true>(part, s); break;
    case 3: rc = launch_tile<LtF3, true>(part, s); break;
    case 4: rc = launch_tile<LtF4, true>(part, s); break;
    case 5: rc = launch_tile<LtF5, true>(part, s); break;
    case 6: rc = launch_tile<LtF6, true>(part, s); break;
    case 7: rc = launch_tile<LtF7, true>(part, s); break;
    default: rc = launch_tile<LtF8, false>(part, s); break;
    }
    if (rc || a.splits == 1)
        return rc;
    a.split_stride = part.split_stride;
    const int64_t total = (int64_t)((a.N + 7) / 8) * a.M;
    const int blocks = (int)std::min<int64_t>((total + 255) / 256, 4096);
    const dim3 grid(blocks + (a.columns.out ? (a.columns.n + 63) / 64 : 0));
    if (a.odt == MOE_DTYPE_F32)
        hipLaunchKernelGGL(linear_join_kernel<float>, grid, dim3(256), 0, s, a,
                           static_cast<const float *>(ws), part.ldo, blocks);
    else
        hipLaunchKernelGGL(linear_join_kernel<f16>, grid, dim3(256), 0, s, a,
                           static_cast<const float *>(ws), part.ldo, blocks);
    MOE_LAUNCH_CHECK("linear_join_kernel");
    return MOE_OK;
}

}  // namespace moe
