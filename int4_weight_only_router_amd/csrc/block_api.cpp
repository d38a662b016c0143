// block_api.cpp -- the C ABI of the operators around a routed block: norms, fp16
// products, balance loss.  Argument validation and dispatch.
#include <cmath>

#include "k_balance.h"
#include "k_linear.h"
#include "trace.h"

namespace moe {

static bool known_type(int dtype)
{
    return dtype == MOE_DTYPE_F16 || dtype == MOE_DTYPE_F32 || dtype == MOE_DTYPE_BF16;
}
static size_t type_size(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

// Whether rows of `size`-byte elements, ld apart, can be read 16 bytes at a time.
static bool rows16(const void *p, int64_t ld, size_t size)
{
    return (uintptr_t)p % 16 == 0 && ld * (int64_t)size % 16 == 0;
}

static int check_norm(const char *fn, const NormArgs &a, int dtype, int w_dtype, int kind,
                      unsigned flags)
{
    if (!known_type(dtype))
        return set_error(MOE_EINVAL, "%s: dtype %d is none of F16, BF16, F32", fn, dtype);
    if (w_dtype != dtype && w_dtype != MOE_DTYPE_F32)
        return set_error(MOE_EINVAL, "%s: weights of dtype %d (F32 or the rows' %d)", fn, w_dtype,
                         dtype);
    if (kind != MOE_NORM_RMS && kind != MOE_NORM_LAYER)
        return set_error(MOE_EINVAL, "%s: unknown norm %d", fn, kind);
    if (flags & ~(unsigned)(MOE_NORM_POST | MOE_NORM_UNIT_OFFSET))
        return set_error(MOE_EINVAL, "%s: unknown flags 0x%x", fn, flags);
    if (a.T < 0 || a.H <= 0)
        return set_error(MOE_EINVAL, "%s: bad sizes T=%d H=%d", fn, a.T, a.H);
    if (!(a.eps >= 0.0f) || !std::isfinite(a.eps) || !std::isfinite(a.scale))
        return set_error(MOE_EINVAL, "%s: eps must be finite and not negative, the scale finite",
                         fn);
    if (a.H > 8192)
        return set_error(MOE_EUNSUPPORTED, "%s: H=%d above 8192", fn, a.H);
    if ((a.gate && a.ldg && a.ldg < a.H) || a.ldg < 0 || (!a.gate && a.ldg))
        return set_error(MOE_EINVAL, "%s: gate stride %lld (0 for one row, else >= H)", fn,
                         (long long)a.ldg);
    if (!a.post && (a.post_w || a.post_b))
        return set_error(MOE_EINVAL, "%s: post-norm weights without MOE_NORM_POST", fn);
    const size_t wa = type_size(w_dtype);
    if ((uintptr_t)a.post_w % wa || (uintptr_t)a.post_b % wa || (uintptr_t)a.pre_w % wa ||
        (uintptr_t)a.pre_b % wa)
        return set_error(MOE_EINVAL, "%s: misaligned weights", fn);
    return MOE_OK;
}

// A row tensor: its stride and alignment.
static int check_rows(const char *fn, const char *what, const void *p, int64_t ld, int H, int dtype)
{
    if (p && (ld < H || (uintptr_t)p % type_size(dtype)))
        return set_error(MOE_EINVAL, "%s: %s: row stride %lld < H=%d, or misaligned", fn, what,
                         (long long)ld, H);
    return MOE_OK;
}

// Whether the rows (of a gradient: those of what it is of) and weights can all be read
// and written 16 bytes at a time.
static bool norm_vec(const NormArgs &a, const NormGrads &d, int dtype)
{
    const size_t s = type_size(dtype);
    const uintptr_t weights = (uintptr_t)a.post_w | (uintptr_t)a.post_b | (uintptr_t)a.pre_w |
                              (uintptr_t)a.pre_b;
    auto rows = [&](const void *p, int64_t ld) { return !p || rows16(p, ld, s); };
    return a.H % 8 == 0 && weights % 16 == 0 && rows(a.y, a.ldy) && rows(d.dy, a.ldy) &&
           rows(a.residual, a.ldr) && rows(d.dresidual, a.ldr) && rows(a.gate, a.ldg) &&
           (!a.ldg || rows(d.dgate, a.ldg)) && rows(a.out, a.ldo) && rows(d.dout, a.ldo) &&
           rows(a.n, a.ldn) && rows(d.dn, a.ldn);
}

static bool known_act(int act) { return act >= MOE_ACT_NONE && act <= MOE_ACT_GELU_TANH; }

static int check_linear(const char *fn, int M, int N, int K, int act, int out_dtype)
{
    if (M < 0 || N <= 0 || K <= 0)
        return set_error(MOE_EINVAL, "%s: bad sizes M=%d N=%d K=%d", fn, M, N, K);
    if (!known_act(act))
        return set_error(MOE_EINVAL, "%s: unknown activation %d", fn, act);
    if (out_dtype != MOE_DTYPE_F16 && out_dtype != MOE_DTYPE_F32)
        return set_error(MOE_EINVAL, "%s: output dtype %d is neither F16 nor F32", fn, out_dtype);
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_block_norm(const void *y, int64_t ldy, const void *residual, int64_t ldr, const void *gate,
                   int64_t ldg, float scale, const void *post_w, const void *post_b,
                   const void *pre_w, const void *pre_b, int dtype, int w_dtype, int kind,
                   unsigned flags, float eps, int T, int H, void *out, int64_t ldo, void *n,
                   int64_t ldn, hipStream_t stream)
{
    MOE_API_RANGE();
    clear_error();
    const char *fn = "moe_block_norm";
    NormArgs a{};
    a.y = y;
    a.residual = residual;
    a.gate = gate;
    a.post_w = post_w;
    a.post_b = post_b;
    a.pre_w = pre_w;
    a.pre_b = pre_b;
    a.out = out;
    a.n = n;
    a.ldy = ldy;
    a.ldr = ldr;
    a.ldg = ldg;
    a.ldo = ldo;
    a.ldn = ldn;
    a.scale = scale;
    a.eps = eps;
    a.T = T;
    a.H = H;
    a.w32 = w_dtype == MOE_DTYPE_F32;
    a.layer = kind == MOE_NORM_LAYER;
    a.post = (flags & MOE_NORM_POST) != 0;
    a.offset = (flags & MOE_NORM_UNIT_OFFSET) != 0;
    int rc = check_norm(fn, a, dtype, w_dtype, kind, flags);
    if (rc || T == 0)
        return rc;
    if ((!y && !residual) || (!out && !n))
        return set_error(MOE_EINVAL, "%s: y or residual, and out or n, are required", fn);
    if (!y && (gate || a.post))
        return set_error(MOE_EINVAL, "%s: a gate or a post norm without y", fn);
    if (!n && (pre_w || pre_b))
        return set_error(MOE_EINVAL, "%s: pre-norm weights without n", fn);
    if ((rc = check_rows(fn, "y", y, ldy, H, dtype)) ||
        (rc = check_rows(fn, "residual", residual, ldr, H, dtype)) ||
        (rc = check_rows(fn, "gate", gate, ldg ? ldg : H, H, dtype)) ||
        (rc = check_rows(fn, "out", out, ldo, H, dtype)) ||
        (rc = check_rows(fn, "n", n, ldn, H, dtype)))
        return rc;
    a.vec = norm_vec(a, NormGrads{}, dtype);
    return launch_block_norm(a, dtype, stream);
}

size_t moe_block_norm_backward_workspace_bytes(int T, int H)
{
    if (T <= 0 || H <= 0 || H > 8192)
        return 0;
    return block_norm_backward_ws(T, H);
}

int moe_block_norm_backward(const void *dout, int64_t ldo, const void *dn, int64_t ldn,
                            const void *y, int64_t ldy, const void *residual, int64_t ldr,
                            const void *gate, int64_t ldg, float scale, const void *post_w,
                            const void *post_b, const void *pre_w, int dtype, int w_dtype, int kind,
                            unsigned flags, float eps, int T, int H, void *dy, void *dresidual,
                            void *dgate, float *dpost_w, float *dpost_b, float *dpre_w,
                            float *dpre_b, void *ws, size_t ws_bytes, hipStream_t stream)
{
    MOE_API_RANGE();
    clear_error();
    const char *fn = "moe_block_norm_backward";
    NormArgs a{};
    a.y = y;
    a.residual = residual;
    a.gate = gate;
    a.post_w = post_w;
    a.post_b = post_b;
    a.pre_w = pre_w;
    a.ldy = ldy;
    a.ldr = ldr;
    a.ldg = ldg;
    a.ldo = ldo;
    a.ldn = ldn;
    a.scale = scale;
    a.eps = eps;
    a.T = T;
    a.H = H;
    a.w32 = w_dtype == MOE_DTYPE_F32;
    a.layer = kind == MOE_NORM_LAYER;
    a.post = (flags & MOE_NORM_POST) != 0;
    a.offset = (flags & MOE_NORM_UNIT_OFFSET) != 0;
    int rc = check_norm(fn, a, dtype, w_dtype, kind, flags);
    if (rc)
        return rc;
    NormGrads d{};
    d.dout = dout;
    d.dn = dn;
    d.dy = dy;
    d.dresidual = dresidual;
    d.dgate = dgate;
    d.sums[0] = ldg == 0 ? static_cast<float *>(dgate) : nullptr;
    d.sums[1] = dpost_w;
    d.sums[2] = dpost_b;
    d.sums[3] = dpre_w;
    d.sums[4] = dpre_b;
    bool any = false;
    for (float *p : d.sums) {
        any |= p != nullptr;
        if ((uintptr_t)p % 4)
            return set_error(MOE_EINVAL, "%s: misaligned fp32 gradients", fn);
    }
    if (T > 0) {
        if ((!y && !residual) || (!dout && !dn))
            return set_error(MOE_EINVAL, "%s: y or residual, and dout or dn, are required", fn);
        if (!y && (gate || a.post || dy || dgate))
            return set_error(MOE_EINVAL, "%s: a gate, a post norm or their gradients without y", fn);
        if (!residual && dresidual)
            return set_error(MOE_EINVAL, "%s: dresidual without residual", fn);
        if (dgate && !gate)
            return set_error(MOE_EINVAL, "%s: dgate without gate", fn);
        if (!dn && (pre_w || dpre_w || dpre_b))
            return set_error(MOE_EINVAL, "%s: pre-norm weights or their gradients without dn", fn);
        if ((dpost_w || dpost_b) && !a.post)
            return set_error(MOE_EINVAL, "%s: post-norm gradients without MOE_NORM_POST", fn);
        if ((rc = check_rows(fn, "dout", dout, ldo, H, dtype)) ||
            (rc = check_rows(fn, "dn", dn, ldn, H, dtype)) ||
            (rc = check_rows(fn, "y", y, ldy, H, dtype)) ||
            (rc = check_rows(fn, "residual", residual, ldr, H, dtype)) ||
            (rc = check_rows(fn, "gate", gate, ldg ? ldg : H, H, dtype)) ||
            (rc = check_rows(fn, "dy", dy, ldy, H, dtype)) ||
            (rc = check_rows(fn, "dresidual", dresidual, ldr, H, dtype)) ||
            (rc = check_rows(fn, "dgate", ldg ? dgate : nullptr, ldg, H, dtype)))
            return rc;
        if (any) {
            const size_t need = moe_block_norm_backward_workspace_bytes(T, H);
            if (!ws || ws_bytes < need)
                return set_error(MOE_ENOMEM, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
            if ((uintptr_t)ws % 16)
                return set_error(MOE_EINVAL, "%s: misaligned workspace", fn);
        }
    }
    d.parts = static_cast<float *>(ws);
    a.vec = norm_vec(a, d, dtype);
    return launch_block_norm_backward(a, d, dtype, stream);
}

size_t moe_linear_f16_workspace_bytes(int M, int N, int K)
{
    if (M <= 0 || N <= 0 || K <= 0)
        return 0;
    const LinPlan p = linear_forward_plan(M, N, K);
    return p.items > LIN_MOST_ITEMS ? 0 : linear_ws(p, M, N);
}

int moe_linear_f16(const void *x_f16, int64_t ldx, const void *w_f16, int64_t ldw,
                   const float *bias, int act, const void *residual, int64_t ldr, int M, int N,
                   int K, void *out, int out_dtype, int64_t ldo, void *z_f16, int64_t ldz, void *ws,
                   size_t ws_bytes, hipStream_t stream)
{
    MOE_API_RANGE();
    clear_error();
    const char *fn = "moe_linear_f16";
    int rc = check_linear(fn, M, N, K, act, out_dtype);
    if (rc)
        return rc;
    if (ldx < K || ldw < K || ldo < N || (residual && ldr < N) || (z_f16 && ldz < N))
        return set_error(MOE_EINVAL, "%s: a row stride is shorter than its row", fn);
    if (K % 8 || ldx % 8 || ldw % 8)
        return set_error(MOE_EUNSUPPORTED,
                         "%s: K, ldx and ldw must be multiples of 8 (K=%d ldx=%lld ldw=%lld)", fn, K,
                         (long long)ldx, (long long)ldw);
    const bool far = ldx > LIN_MOST_LD || ldw > LIN_MOST_LD;
    const LinPlan plan = far || M == 0 ? LinPlan{} : linear_forward_plan(M, N, K);
    if (far || plan.items > LIN_MOST_ITEMS)
        return set_error(MOE_EUNSUPPORTED,
                         "%s: rows of at most %d elements and %lld tiles (M=%d N=%d ldx=%lld "
                         "ldw=%lld)", fn, LIN_MOST_LD, (long long)LIN_MOST_ITEMS, M, N,
                         (long long)ldx, (long long)ldw);
    if (M == 0)
        return MOE_OK;
    if (!x_f16 || !w_f16 || !out)
        return set_error(MOE_EINVAL, "%s: null pointer", fn);
    if (((uintptr_t)x_f16 | (uintptr_t)w_f16) & 15u)
        return set_error(MOE_EINVAL, "%s: x and w must be 16-byte aligned", fn);
    if ((uintptr_t)bias % 4 || (uintptr_t)z_f16 % 2 ||
        ((uintptr_t)out | (uintptr_t)residual) % type_size(out_dtype))
        return set_error(MOE_EINVAL, "%s: misaligned bias, residual, out or z", fn);
    const size_t need = linear_ws(plan, M, N);
    if (need && (!ws || ws_bytes < need))
        return set_error(MOE_ENOMEM, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
    if (need && (uintptr_t)ws % 16)
        return set_error(MOE_EINVAL, "%s: misaligned workspace", fn);
    LinArgs a{};
    a.a = static_cast<const f16 *>(x_f16);
    a.lda = ldx;
    a.b = static_cast<const f16 *>(w_f16);
    a.ldb = ldw;
    a.M = M;
    a.N = N;
    a.K = K;
    a.bias = bias;
    a.act = act;
    a.residual = residual;
    a.ldr = ldr;
    a.out = out;
    a.odt = out_dtype;
    a.ldo = ldo;
    a.z = static_cast<f16 *>(z_f16);
    a.ldz = ldz;
    return launch_linear(a, plan, ws, stream);
}

size_t moe_linear_f16_backward_workspace_bytes(int M, int N, int K)
{
    if (M <= 0 || N <= 0 || K <= 0)
        return 0;
    const LinGradPlan p = linear_grad_plan(M, N, K);
    return p.fits ? (size_t)p.total : 0;
}

int moe_linear_f16_backward(const void *dy_f16, int64_t lddy, const void *z_f16, int64_t ldz,
                            int act, const void *x_f16, int64_t ldx, const void *w_f16, int64_t ldw,
                            int M, int N, int K, void *dx, int64_t lddx, void *dw, int64_t lddw,
                            int out_dtype, float *dbias, void *ws, size_t ws_bytes,
                            hipStream_t stream)
{
    MOE_API_RANGE();
    clear_error();
    const char *fn = "moe_linear_f16_backward";
    const bool rounded = out_dtype & MOE_DZ_F16;
    out_dtype &= ~MOE_DZ_F16;
    int rc = check_linear(fn, M, N, K, act, out_dtype);
    if (rc)
        return rc;
    if (lddy < N || (act != MOE_ACT_NONE && ldz < N) || (dw && ldx < K) || (dx && ldw < K) ||
        (dx && lddx < K) || (dw && lddw < K))
        return set_error(MOE_EINVAL, "%s: a row stride is shorter than its row", fn);
    if (K % 8 || (dw && ldx % 8) || (dx && ldw % 8))
        return set_error(MOE_EUNSUPPORTED,
                         "%s: K, ldx and ldw must be multiples of 8 (K=%d ldx=%lld ldw=%lld)", fn, K,
                         (long long)ldx, (long long)ldw);
    const bool far = (dw && ldx > LIN_MOST_LD) || (dx && ldw > LIN_MOST_LD) || N > LIN_MOST_LD;
    const bool two = !rounded && !linear_dz_exact(act);
    const LinGradPlan plan = far || M == 0 ? LinGradPlan{} : linear_grad_plan(M, N, K);
    if (far || (M > 0 && !(two ? plan.fits2 : plan.fits)))
        return set_error(MOE_EUNSUPPORTED,
                         "%s: rows of at most %d elements and %lld tiles (M=%d N=%d K=%d ldx=%lld "
                         "ldw=%lld)", fn, LIN_MOST_LD, (long long)LIN_MOST_ITEMS, M, N, K,
                         (long long)ldx, (long long)ldw);
    if (act != MOE_ACT_NONE && out_dtype == MOE_DTYPE_F32)
        return set_error(MOE_EUNSUPPORTED,
                         "%s: fp32 gradients through an activation", fn);
    if (!dx && !dw && !dbias)
        return set_error(MOE_EINVAL, "%s: no gradient asked for", fn);
    if (M > 0 && (!dy_f16 || (act != MOE_ACT_NONE && !z_f16) || (dw && !x_f16) || (dx && !w_f16)))
        return set_error(MOE_EINVAL, "%s: null pointer", fn);
    if (((dw ? (uintptr_t)x_f16 : 0) | (dx ? (uintptr_t)w_f16 : 0)) & 15u)
        return set_error(MOE_EINVAL, "%s: x and w must be 16-byte aligned", fn);
    if ((uintptr_t)dy_f16 % 2 || (act != MOE_ACT_NONE && (uintptr_t)z_f16 % 2) ||
        (uintptr_t)dbias % 4 || ((uintptr_t)dx | (uintptr_t)dw) % type_size(out_dtype))
        return set_error(MOE_EINVAL, "%s: misaligned dy, z or gradients", fn);
    const size_t need = (size_t)plan.total;
    if (need && (!ws || ws_bytes < need))
        return set_error(MOE_ENOMEM, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
    if (need && (uintptr_t)ws % 16)
        return set_error(MOE_EINVAL, "%s: misaligned workspace", fn);
    LinGrads g{};
    g.dy = static_cast<const f16 *>(dy_f16);
    g.lddy = lddy;
    g.z = static_cast<const f16 *>(z_f16);
    g.ldz = ldz;
    g.act = act;
    g.x = static_cast<const f16 *>(x_f16);
    g.ldx = ldx;
    g.w = static_cast<const f16 *>(w_f16);
    g.ldw = ldw;
    g.M = M;
    g.N = N;
    g.K = K;
    g.dx = dx;
    g.lddx = lddx;
    g.dw = dw;
    g.lddw = lddw;
    g.odt = out_dtype;
    g.two = two;
    g.dbias = dbias;
    return launch_linear_backward(g, plan, ws, stream);
}

size_t moe_balance_loss_workspace_bytes(int T, int E)
{
    return T <= 0 || E <= 0 || E > BL_MAX_E ? 0 : balance_ws(T, E);
}

int moe_balance_loss(const void *logits, int logits_dtype, int64_t ld, const int32_t *topk_idx,
                     const uint8_t *token_mask, int T, int E, int k, int score, float coef,
                     float z_coef, int32_t *counts, float *mean_prob, float *losses,
                     const float *d_loss, void *dlogits, int dlogits_dtype, int64_t ldd, void *ws,
                     size_t ws_bytes, hipStream_t stream)
{
    MOE_API_RANGE();
    clear_error();
    const char *fn = "moe_balance_loss";
    if (T < 0 || E <= 0 || k <= 0 || k > E)
        return set_error(MOE_EINVAL, "%s: need T >= 0, E > 0, 0 < k <= E (T=%d E=%d k=%d)", fn, T,
                         E, k);
    if (!known_type(logits_dtype) || (dlogits && !known_type(dlogits_dtype)))
        return set_error(MOE_EINVAL, "%s: dtypes %d, %d (F16, BF16 or F32)", fn, logits_dtype,
                         dlogits_dtype);
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
        return set_error(MOE_EINVAL, "%s: unknown score function %d", fn, score);
    if (!std::isfinite(coef) || !std::isfinite(z_coef))
        return set_error(MOE_EINVAL, "%s: a coefficient is not finite", fn);
    if (ld < E || (dlogits && ldd < E))
        return set_error(MOE_EINVAL, "%s: row strides %lld, %lld < E=%d", fn, (long long)ld,
                         (long long)ldd, E);
    if (E > BL_MAX_E)
        return set_error(MOE_EUNSUPPORTED, "%s: E=%d above %d", fn, E, BL_MAX_E);
    if ((int64_t)T * k >= (int64_t)1 << 31)
        return set_error(MOE_EUNSUPPORTED, "%s: T*k too large", fn);
    if (!counts || (T > 0 && !logits))
        return set_error(MOE_EINVAL, "%s: null pointer", fn);
    if ((uintptr_t)logits % type_size(logits_dtype) ||
        (dlogits && (uintptr_t)dlogits % type_size(dlogits_dtype)) ||
        ((uintptr_t)topk_idx | (uintptr_t)counts | (uintptr_t)mean_prob | (uintptr_t)losses |
         (uintptr_t)d_loss) % 4)
        return set_error(MOE_EINVAL, "%s: misaligned pointer", fn);
    const size_t need = moe_balance_loss_workspace_bytes(T, E);
    if (need && (!ws || ws_bytes < need))
        return set_error(MOE_ENOMEM, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
    if (need && (uintptr_t)ws % 16)
        return set_error(MOE_EINVAL, "%s: misaligned workspace", fn);
    BalanceArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.idx = topk_idx;
    a.mask = token_mask;
    a.T = T;
    a.E = E;
    a.k = k;
    a.score = score;
    a.coef = coef;
    a.zcoef = z_coef;
    a.counts = counts;
    a.mean_prob = mean_prob;
    a.losses = losses;
    a.d_loss = d_loss;
    a.dlogits = dlogits;
    a.gtype = dlogits_dtype;
    a.ldd = ldd;
    return launch_balance(a, logits_dtype, ws, stream);
}

}  // extern "C"
