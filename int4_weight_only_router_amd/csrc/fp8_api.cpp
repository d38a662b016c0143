// fp8_api.cpp -- the C ABI of score routing and of the block-scaled FP8
// operators: argument validation, choice of kernel, dispatch.
#include <algorithm>
#include <cmath>

#include "k_fp8_frag.h"
#include "trace.h"

namespace moe {

int launch_route_batched_logits(const void *, const void *, const float *, int, int, int, float *,
                                hipStream_t);
int launch_route_logits_rows(const void *, const void *, const float *, int, int, int, float *,
                             hipStream_t);
size_t route_select_ws_bytes(int T, int k, int E);
int launch_route_select(const void *, int, int64_t, const float *, int, int, int, int, int, int,
                        unsigned, float, int32_t *, float *, int32_t *, int32_t *, int32_t *,
                        int32_t *, void *, hipStream_t);
int launch_quant_fp8(const void *, int, int64_t, int64_t, int, int, bool, void *, int64_t, float *,
                     hipStream_t);
int launch_fp8_tokens(const void *, int64_t, int, uint8_t *, float *, const int32_t *,
                      const void *const *, int, int, Fp8TileRec *, hipStream_t);
int launch_fp8_rows_dense(const Fp8Args &, hipStream_t);
int launch_fp8_tile_dense(const Fp8Args &, int mf, bool acc32, hipStream_t);
int launch_fp8_decode(Fp8Args, const void *, float *, int, int, const int64_t *, void *,
                      hipStream_t);
int fp8_pick_rows(int64_t rows, int E, int I);
int64_t fp8_tile_bound(int64_t rows, int E, int bm);
int64_t fp8_most_tiles(int64_t rows, int H, int I, int E);
int launch_fp8_experts(Fp8Args, int, uint8_t *, float *, int, int, const int64_t *, void *,
                       bool acc32, hipStream_t);

static int check_types(const char *fn, int dtype)
{
    if (dtype != MOE_DTYPE_F16 && dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
        return set_error(MOE_EINVAL, "%s: dtype %d is none of F16, BF16, F32", fn, dtype);
    return MOE_OK;
}

static size_t dtype_size(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

// Canonical FP8 blob sections (documented in moe_w4a16.h).
static void fp8_blob(int H, int I, int64_t off[6], int64_t *total)
{
    const int64_t w = (int64_t)I * H;
    const int64_t s = (int64_t)((I + 127) / 128) * ((H + 127) / 128) * 4;
    int64_t o = 0;
    for (int i = 0; i < 6; ++i) {
        off[i] = o;
        o = al256(o + (i < 3 ? w : s));
    }
    *total = o;
}

static int check_fp8_shape(const char *fn, int T, int H, int I, int E, int k)
{
    if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0 || k > E)
        return set_error(MOE_EINVAL, "%s: bad sizes T=%d H=%d I=%d E=%d k=%d", fn, T, H, I, E, k);
    if (H % 64 || I % 64 || H > 8192 || I > 8192 || E > 1024 || k > 16)
        return set_error(MOE_EUNSUPPORTED,
                         "%s: H and I multiples of 64 up to 8192, E <= 1024, k <= 16 required "
                         "(H=%d I=%d E=%d k=%d)", fn, H, I, E, k);
    if ((int64_t)T * k >= (int64_t)1 << 31)
        return set_error(MOE_EUNSUPPORTED, "%s: T*k too large", fn);
    return MOE_OK;
}

// Workspace of the routed FP8 experts.
struct Fp8Ws {
    int64_t xq, xs, hq, hs, tiles, h, total;
};
static Fp8Ws fp8_ws(int T, int H, int I, int E, int k, bool decode)
{
    Fp8Ws w{};
    const int64_t n = (int64_t)T * k;
    int64_t o = 0;
    if (decode) {
        w.h = o;
        o = al256(o + n * I * 4);
    } else {
        w.xq = o;    o = al256(o + (int64_t)T * H);
        w.xs = o;    o = al256(o + (int64_t)T * ((H + 127) / 128) * 4);
        w.hq = o;    o = al256(o + n * I);
        w.hs = o;    o = al256(o + n * ((I + 127) / 128) * 4);
        w.tiles = o; o = al256(o + (1 + fp8_tile_bound(n, E, fp8_pick_rows(n, E, I))) * sizeof(Fp8TileRec));
    }
    w.total = o;
    return w;
}

// Kernel of a dense product: 64*mf x 256 tiles, or 0 for the kernel of few rows
// (32 x 32 tiles).  The least of the times that were measured for one round of
// tiles over the 256 compute units at K = 2048 (every form grows alike with K),
// in us: 64-, 128-, 192- and 256-row tiles 14.5, 20.5, 24.5, 29.5, and 24, 33.5,
// 43, 52.5 in the fp16 form (fp32 outputs or sums); the kernel of few rows 2.5 and 9.8
// for every 1000 workgroups.  Against each form on 28 products from 64 x 5632 to
// 4096 x 11264 (K 512 to 5632, both forms) the choice is the fastest or within
// 3% of it.
static int dense_tile(int M, int N, bool f16_form)
{
    static const double round_us[2][4] = {{14.5, 20.5, 24.5, 29.5}, {24, 33.5, 43, 52.5}};
    const int64_t few = (int64_t)((M + 31) / 32) * ((N + 31) / 32);
    double best = 2.5 + 9.8e-3 * (double)few;
    int mf = 0;
    for (int i = 1; i <= 4; ++i) {
        const int64_t tiles = (int64_t)((M + 64 * i - 1) / (64 * i)) * ((N + 255) / 256);
        const double t = 3 + (double)((tiles + 255) / 256) * (round_us[f16_form][i - 1] - 3);
        if (M > 32 && t < best) {
            best = t;
            mf = i;
        }
    }
    return mf;
}

static int check_select(const char *fn, const void *logits, int dtype, int64_t ld, int T, int E,
                        int k, int score, int n_group, int topk_group, unsigned flags, float scale,
                        const float *bias, const int32_t *topk_idx, const float *topk_w)
{
    if (T < 0 || E <= 0 || k <= 0 || k > E)
        return set_error(MOE_EINVAL, "%s: need T >= 0, E > 0, 0 < k <= E (T=%d E=%d k=%d)", fn, T,
                         E, k);
    int rc = check_types(fn, dtype);
    if (rc)
        return rc;
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
        return set_error(MOE_EINVAL, "%s: unknown score function %d", fn, score);
    if (flags & ~(unsigned)(MOE_RENORM | MOE_GROUP_TOP2))
        return set_error(MOE_EINVAL, "%s: unknown flags 0x%x", fn, flags);
    if (n_group <= 0 || E % n_group || topk_group <= 0 || topk_group > n_group)
        return set_error(MOE_EINVAL, "%s: %d groups (%d kept) of %d experts", fn, n_group,
                         topk_group, E);
    if ((int64_t)topk_group * (E / n_group) < k)
        return set_error(MOE_EINVAL, "%s: %d kept groups of %d experts hold fewer than k=%d", fn,
                         topk_group, E / n_group, k);
    if (ld < E)
        return set_error(MOE_EINVAL, "%s: row stride %lld < E=%d", fn, (long long)ld, E);
    if (!std::isfinite(scale))
        return set_error(MOE_EINVAL, "%s: the scale is not finite", fn);
    if (E > 1024 || k > 16 || n_group > 64)
        return set_error(MOE_EUNSUPPORTED,
                         "%s: E <= 1024, k <= 16 and at most 64 groups required (E=%d k=%d "
                         "groups=%d)", fn, E, k, n_group);
    if (T > 1 << 25)   // a wave per token, and a launch has fewer than 2^32 threads
        return set_error(MOE_EUNSUPPORTED, "%s: T=%d above 2^25", fn, T);
    if (T > 0 && (!logits || !topk_idx || !topk_w))
        return set_error(MOE_EINVAL, "%s: null pointer", fn);
    if ((uintptr_t)logits % dtype_size(dtype) ||
        ((uintptr_t)bias | (uintptr_t)topk_idx | (uintptr_t)topk_w) % 4)
        return set_error(MOE_EINVAL, "%s: misaligned pointer", fn);
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_router_logits(const void *x_f16, const void *w_router_f16, const float *logit_bias, int T,
                      int H, int E, float *logits, hipStream_t stream)
{
    MOE_API_RANGE();
    clear_error();
    const char *fn = "moe_router_logits";
    if (T < 0 || H <= 0 || H % 8 || E <= 0)
        return set_error(MOE_EINVAL, "%s: bad shape T=%d H=%d E=%d", fn, T, H, E);
    if (!h_supported(H) || E > 1024)
        return set_error(MOE_EUNSUPPORTED, "%s: H in {256, 512, 1024, 2048} and E <= 1024 required "
                         "(H=%d E=%d)", fn, H, E);
    if (T > (1 << 27) - 8)   // 256 threads for 8 tokens, and a launch has fewer than 2^32
        return set_error(MOE_EUNSUPPORTED, "%s: T=%d above 2^27 - 8", fn, T);
    if (T == 0)
        return MOE_OK;
    if (!x_f16 || !w_router_f16 || !logits)
        return set_error(MOE_EINVAL, "%s: null pointer", fn);
    if (((uintptr_t)x_f16 | (uintptr_t)w_router_f16) & 15u)
        return set_error(MOE_EINVAL, "%s: x and the router must be 16-byte aligned", fn);
    if (T <= 4)
        return launch_route_logits_rows(x_f16, w_router_f16, logit_bias, T, H, E, logits, stream);
    return launch_route_batched_logits(x_f16, w_router_f16, logit_bias, T, H, E, logits, stream);
}

int moe_route_select(const void *logits, int logits_dtype, int64_t ld, const float *select_bias,
                     int T, int E, int k, int score, int n_group, int topk_group, unsigned flags,
                     float scale, int32_t *topk_idx, float *topk_w, hipStream_t stream)
{
    MOE_API_RANGE();
    clear_error();
    const int rc = check_select("moe_route_select", logits, logits_dtype, ld, T, E, k, score,
                                n_group, topk_group, flags, scale, select_bias, topk_idx, topk_w);
    if (rc || T == 0)
        return rc;
    return launch_route_select(logits, logits_dtype, ld, select_bias, T, E, k, score, n_group,
                               topk_group, flags, scale, topk_idx, topk_w, nullptr, nullptr,
                               nullptr, nullptr, nullptr, stream);
}

size_t moe_route_select_workspace_bytes(int T, int k, int E)
{
    if (T < 0 || k <= 0 || E <= 0)
        return 0;
    return route_select_ws_bytes(T, k, E);
}

int moe_route_select_permute(const void *logits, int logits_dtype, int64_t ld,
                             const float *select_bias, int T, int E, int k, int score, int n_group,
                             int topk_group, unsigned flags, float scale, int32_t *topk_idx,
                             float *topk_w, int32_t *counts, int32_t *offsets, int32_t *perm,
                             int32_t *inv_perm, void *ws, size_t ws_bytes, hipStream_t stream)
{
    MOE_API_RANGE();
    clear_error();
    const char *fn = "moe_route_select_permute";
    int rc = check_select(fn, logits, logits_dtype, ld, T, E, k, score, n_group, topk_group, flags,
                          scale, select_bias, topk_idx, topk_w);
    if (rc)
        return rc;
    if (!counts || !offsets || (T > 0 && (!perm || !inv_perm)))
        return set_error(MOE_EINVAL, "%s: null pointer", fn);
    if (((uintptr_t)counts | (uintptr_t)offsets | (uintptr_t)perm | (uintptr_t)inv_perm) % 4)
        return set_error(MOE_EINVAL, "%s: misaligned pointer", fn);
    const size_t need = moe_route_select_workspace_bytes(T, k, E);
    if (need && (!ws || ws_bytes < need))
        return set_error(MOE_ENOMEM, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
    if (need && (uintptr_t)ws % 16)
        return set_error(MOE_EINVAL, "%s: misaligned workspace", fn);
    return launch_route_select(logits, logits_dtype, ld, select_bias, T, E, k, score, n_group,
                               topk_group, flags, scale, topk_idx, topk_w, counts, offsets, perm,
                               inv_perm, ws, stream);
}

int moe_quantize_fp8(const void *x, int dtype, int64_t ldx, int64_t rows, int cols, int block_rows,
                     unsigned flags, void *q, int64_t ldq, float *scales, hipStream_t stream)
{
    MOE_API_RANGE();
    clear_error();
    const char *fn = "moe_quantize_fp8";
    int rc = check_types(fn, dtype);
    if (rc)
        return rc;
    if (rows < 0 || cols <= 0 || ldx < cols || ldq < cols)
        return set_error(MOE_EINVAL, "%s: bad sizes rows=%lld cols=%d ldx=%lld ldq=%lld", fn,
                         (long long)rows, cols, (long long)ldx, (long long)ldq);
    if (block_rows != 1 && block_rows != 128)
        return set_error(MOE_EINVAL, "%s: blocks of %d rows (1 or 128)", fn, block_rows);
    if (flags & ~(unsigned)MOE_SCALE_POW2)
        return set_error(MOE_EINVAL, "%s: unknown flags 0x%x", fn, flags);
    // a row of blocks must fit one launch, and the blocks' number 64 bits
    if (cols > 1 << 30 || rows > (1LL << 36) / ((cols + 127) / 128))
        return set_error(MOE_EUNSUPPORTED, "%s: rows=%lld cols=%d", fn, (long long)rows, cols);
    if (rows == 0)
        return MOE_OK;
    if (!x || !q || !scales)
        return set_error(MOE_EINVAL, "%s: null pointer", fn);
    if ((uintptr_t)x % dtype_size(dtype) || (uintptr_t)scales % 4)
        return set_error(MOE_EINVAL, "%s: misaligned x or scales", fn);
    return launch_quant_fp8(x, dtype, ldx, rows, cols, block_rows, (flags & MOE_SCALE_POW2) != 0, q,
                            ldq, scales, stream);
}

int moe_gemm_fp8(const void *xq, int64_t ldx, const float *x_scales, const void *wq, int64_t ldw,
                 const float *w_scales, int M, int N, int K, void *out, int out_dtype, int64_t ldo,
                 hipStream_t stream)
{
    MOE_API_RANGE();
    clear_error();
    const char *fn = "moe_gemm_fp8";
    const bool acc32 = (out_dtype & MOE_ACC_F32) != 0;
    out_dtype &= ~MOE_ACC_F32;
    int rc = check_types(fn, out_dtype);
    if (rc)
        return rc;
    if (M < 0 || N <= 0 || K <= 0 || ldx < K || ldw < K || ldo < N)
        return set_error(MOE_EINVAL, "%s: bad sizes M=%d N=%d K=%d ldx=%lld ldw=%lld ldo=%lld", fn,
                         M, N, K, (long long)ldx, (long long)ldw, (long long)ldo);
    if (K % 16 || K > 16384 || ldx % 16 || ldw % 16)
        return set_error(MOE_EUNSUPPORTED,
                         "%s: K (at most 16384), ldx and ldw must be multiples of 16 (K=%d "
                         "ldx=%lld ldw=%lld)", fn, K, (long long)ldx, (long long)ldw);
    if (M > 0x7fffff00 || N > 0x7fffff00)   // whole tiles stay within an int
        return set_error(MOE_EUNSUPPORTED, "%s: M=%d N=%d", fn, M, N);
    if (M == 0)
        return MOE_OK;
    if (!xq || !x_scales || !wq || !w_scales || !out)
        return set_error(MOE_EINVAL, "%s: null pointer", fn);
    if ((((uintptr_t)xq | (uintptr_t)wq) & 15u) || ((uintptr_t)x_scales | (uintptr_t)w_scales) % 4 ||
        (uintptr_t)out % dtype_size(out_dtype))
        return set_error(MOE_EINVAL, "%s: xq and wq must be 16-byte aligned, scales and out to "
                         "their elements", fn);
    Fp8Args a{};
    a.x = static_cast<const uint8_t *>(xq);
    a.xs = x_scales;
    a.ldx = ldx;
    a.w = static_cast<const uint8_t *>(wq);
    a.ws = w_scales;
    a.ldw = ldw;
    a.M = M;
    a.N = N;
    a.K = K;
    a.out = out;
    a.ldo = ldo;
    a.odt = out_dtype;
    const int mf = dense_tile(M, N, acc32 || out_dtype == MOE_DTYPE_F32);
    // (the tile kernel's offsets inside 256 weight rows are 32 bits wide)
    const bool few_rows = (M + 31) / 32 <= 65535 && N <= 1 << 28;   // its grid's limits
    if (ldw < (int64_t)1 << 22 && (mf || !few_rows))
        return launch_fp8_tile_dense(a, mf ? mf : 4, acc32, stream);
    if (!few_rows)
        return set_error(MOE_EUNSUPPORTED, "%s: M=%d N=%d with ldw=%lld", fn, M, N,
                         (long long)ldw);
    return launch_fp8_rows_dense(a, stream);
}

int moe_fp8_blob_layout(int H, int I, int64_t offsets[6], int64_t *total_bytes)
{
    clear_error();
    if (!offsets || !total_bytes || H <= 0 || I <= 0)
        return set_error(MOE_EINVAL, "moe_fp8_blob_layout: bad arguments (H=%d I=%d)", H, I);
    if (H > 1 << 30 || I > 1 << 30)   // three H x I sections fit 63 bits
        return set_error(MOE_EUNSUPPORTED, "moe_fp8_blob_layout: H=%d I=%d above 2^30", H, I);
    fp8_blob(H, I, offsets, total_bytes);
    return MOE_OK;
}

int moe_expert_ffn_w8a8_plan(int T, int H, int I, int E, int k, int regime, int *resolved_regime,
                             size_t *ws_bytes)
{
    clear_error();
    const char *fn = "moe_expert_ffn_w8a8_plan";
    const int rc = check_fp8_shape(fn, T, H, I, E, k);
    if (rc)
        return rc;
    const int acc32 = regime & MOE_ACC_F32;
    regime &= ~MOE_ACC_F32;
    if (regime != MOE_REGIME_AUTO && regime != MOE_REGIME_DECODE && regime != MOE_REGIME_BATCHED)
        return set_error(MOE_EINVAL, "%s: bad regime %d", fn, regime);
    // decode up to 64 routed rows, and up to 192 of short tokens, where its one
    // launch less counts more than quantising a token in every workgroup
    // (measured, us decode / batched: H = 2048, 64 experts, top-8, 1 token 15 /
    // 32, 4: 32 / 36, 8: 48 / 64, 12: 73 / 75, 16: 92 / 78; 60 experts, top-4,
    // 8: 41 / 60, 16: 77 / 74; 8 experts, top-2, 16: 19 / 31; H = 1024, 96 rows
    // over 82 experts of I = 384: 28 / 29, 192 over 59 of 768: 39 / 36; H = 512,
    // 192 over 16 of 256: 12 / 15, 480 over 24 of 64: 20 / 18; H = 256, 192 over
    // 97 of 512: 20 / 22, 320 over 12 of 768: 21 / 17)
    const bool fits = T <= FP8_DECODE_MAX_T &&
                      std::min(T, FP8_DECODE_ROWS) * ((std::max(H, I) + 127) / 128) <=
                          FP8_DECODE_BLOCKS;
    const int64_t n = (int64_t)T * k;
    const bool few = n <= 64 || (n <= 192 && n * ((H + 127) / 128) <= 1024);
    const int r = regime != MOE_REGIME_AUTO ? regime
                  : fits && few             ? MOE_REGIME_DECODE
                                            : MOE_REGIME_BATCHED;
    if (r == MOE_REGIME_DECODE && !fits)
        return set_error(MOE_EUNSUPPORTED,
                         "%s: the decode regime takes T <= %d and min(T, %d) * ceil(max(H, I) / "
                         "128) <= %d (T=%d H=%d I=%d)", fn, FP8_DECODE_MAX_T, FP8_DECODE_ROWS,
                         FP8_DECODE_BLOCKS, T, H, I);
    // what the batched launches hold; here, so that nothing is launched beyond it
    if (r == MOE_REGIME_BATCHED && ((int64_t)T * ((H + 127) / 128) > FP8_MOST_TOKEN_BLOCKS ||
                                    fp8_most_tiles(n, H, I, E) > FP8_MOST_TILES))
        return set_error(MOE_EUNSUPPORTED,
                         "%s: more than %d token blocks or %d tiles (T=%d H=%d I=%d E=%d k=%d)", fn,
                         FP8_MOST_TOKEN_BLOCKS, FP8_MOST_TILES, T, H, I, E, k);
    if (resolved_regime)
        *resolved_regime = r | acc32;
    if (ws_bytes)
        *ws_bytes = (size_t)fp8_ws(T, H, I, E, k, r == MOE_REGIME_DECODE).total;
    return MOE_OK;
}

int moe_expert_ffn_w8a8(const void *x_f16, const int32_t *perm, const int32_t *offsets,
                        const void *const *d_expert_blobs, int T, int H, int I, int E, int k,
                        int regime, void *y_f16, void *ws, size_t ws_bytes, hipStream_t stream)
{
    MOE_API_RANGE();
    const char *fn = "moe_expert_ffn_w8a8";
    int r = 0;
    size_t need = 0;
    int rc = moe_expert_ffn_w8a8_plan(T, H, I, E, k, regime, &r, &need);
    if (rc || T == 0)
        return rc;
    if (!x_f16 || !perm || !offsets || !d_expert_blobs || !y_f16)
        return set_error(MOE_EINVAL, "%s: null pointer", fn);
    if (((uintptr_t)x_f16 | (uintptr_t)y_f16 | (uintptr_t)ws) & 15u)
        return set_error(MOE_EINVAL, "%s: x, y and the workspace must be 16-byte aligned", fn);
    if (!ws || ws_bytes < need)
        return set_error(MOE_ENOMEM, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
    const bool decode = (r & ~MOE_ACC_F32) == MOE_REGIME_DECODE;
    const Fp8Ws w = fp8_ws(T, H, I, E, k, decode);
    uint8_t *base = static_cast<uint8_t *>(ws);
    int64_t off[6], total = 0;
    fp8_blob(H, I, off, &total);
    Fp8Args a{};
    a.blobs = d_expert_blobs;
    a.offsets = offsets;
    a.perm = perm;
    a.E = E;
    a.k = k;
    a.T = T;
    if (decode)
        return launch_fp8_decode(a, x_f16, reinterpret_cast<float *>(base + w.h), H, I, off, y_f16,
                                 stream);
    const int64_t n = (int64_t)T * k;
    const int bm = fp8_pick_rows(n, E, I);
    Fp8TileRec *tiles = reinterpret_cast<Fp8TileRec *>(base + w.tiles);
    float *xs = reinterpret_cast<float *>(base + w.xs);
    rc = launch_fp8_tokens(x_f16, T, H, base + w.xq, xs, offsets, d_expert_blobs, E, bm, tiles,
                           stream);
    if (rc)
        return rc;
    a.x = base + w.xq;
    a.xs = xs;
    a.tiles = tiles;
    return launch_fp8_experts(a, bm, base + w.hq, reinterpret_cast<float *>(base + w.hs), H, I, off,
                              y_f16, (r & MOE_ACC_F32) != 0, stream);
}

}  // extern "C"
