/*
 * moe_w4a16.h -- C ABI of libmoe_w4a16.so, the MI355X (gfx950) hot path of a
 * sparsely-activated Mixture-of-Experts layer with INT4 weight-only routed
 * experts and FP16 activations (W4A16).
 *
 * Sources.  The pages describe the method, not an API:
 *  - Horizon RunMap, "Prévia Técnica" (horizonrunmap.com/pt):
 *    "02 / A solução", "03 / Arquitetura" -- the router chooses experts; own
 *    kernels combine compact INT4 weights and FP16 scales with FP16
 *    activations and hand the result back to the model, never keeping an
 *    expanded expert; non-routed parts stay FP16; the optional slot cache
 *    (resident-qpacked-cache-v1) with an immutable host source, temporary
 *    slots, generation publish and consumer retirement.
 *    "08 / Comportamento do modelo" -- W4 = INT4 expert weights with FP16
 *    scales, A16 = FP16 activations, FP32 accumulation stages with explicit
 *    roundings.
 *  - Hamidun News, "Desenvolvedor do Strata cria mapa ao vivo de 24 576
 *    especialistas MoE em uma GTX 1070", "Como 125 bilhões de parâmetros
 *    cabem em 8 GB" -- hot experts resident, the rest loaded on demand,
 *    eviction by an access counter with decay.
 * Where the pages are silent (softmax form, tie-break, SwiGLU, group size,
 * quantiser rounding, logit summation order, eviction constants) the
 * functions follow fixed readings stated next to each declaration.
 *
 * Conventions
 *  - Every function returns MOE_OK (0) or a negative MOE_E* code; a
 *    thread-local message is available from moe_last_error().  No exception
 *    crosses the ABI.
 *  - Shapes and pointers are validated on the host before anything is
 *    launched; on error nothing is launched and outputs are untouched.
 *  - "device" pointers are HIP device memory (hipMalloc / torch CUDA
 *    tensors) of the current device; "host" pointers are CPU memory.
 *  - The caller allocates and owns every activation, weight, output and
 *    workspace; compute calls never allocate.  The slot pool owns its HBM
 *    slots, tables, side stream and events (allocated once at creation).
 *  - Compute calls are asynchronous on the caller's stream and do not
 *    synchronise with the host.  Inputs must be finite (not checked).
 *  - Layouts are row-major; fp16 is IEEE binary16; int32 indices.
 *
 * Kernel envelope (MOE_EUNSUPPORTED outside it): H in {256, 512, 1024, 2048};
 * I a multiple of 64 (up to 8192); group g in {32, 64, 128} dividing
 * H and I; E <= 1024; k <= 16 and k <= E; T*k < 2^31.
 */
#ifndef MOE_W4A16_H
#define MOE_W4A16_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ codes */
enum {
    MOE_OK = 0,
    MOE_EINVAL = -1,        /* null pointer, bad size, k > E, g does not divide H/I ... */
    MOE_EUNSUPPORTED = -2,  /* valid but outside the kernel envelope */
    MOE_ENOMEM = -3,        /* workspace too small, or pool allocation failed */
    MOE_EHIP = -4,          /* a HIP runtime call failed (message has the hipError_t) */
    MOE_ECAPACITY = -5,     /* the slot pool rejects the profile or the routed set */
    MOE_ESTATE = -6         /* slot pool used out of order */
};

enum { MOE_RENORM = 1u };                       /* moe_route flag */
enum { MOE_GROUP_TOP2 = 2u };                   /* moe_route_select flag */
enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };
enum { MOE_SCALE_POW2 = 1u };                   /* moe_quantize_fp8 flag */
enum { MOE_NORM_RMS = 0, MOE_NORM_LAYER = 1 };
/* moe_block_norm flags: the block's output is normed too; weights count as 1 + w */
enum { MOE_NORM_POST = 1u, MOE_NORM_UNIT_OFFSET = 2u };
/* activations of moe_linear_f16; GELU by the error function, GELU_TANH by its
 * tanh form */
enum { MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2, MOE_ACT_GELU = 3,
       MOE_ACT_GELU_TANH = 4 };
/* OR'd into out_dtype of moe_linear_f16_backward: dz is rounded to fp16. */
enum { MOE_DZ_F16 = 0x1000 };
/* OR'd into out_dtype of moe_gemm_fp8 and into the regime of
 * moe_expert_ffn_w8a8(_plan): every sum has fp32 accuracy, whatever the sizes. */
enum { MOE_ACC_F32 = 0x800 };
enum { MOE_REGIME_AUTO = 0, MOE_REGIME_DECODE = 1, MOE_REGIME_BATCHED = 2, MOE_REGIME_SMALL = 3 };
/* OR'd into the regime of moe_expert_ffn_plan / moe_expert_ffn_w4a16: y rows
 * in token order (row t*k + j) instead of sorted order; see below. */
enum { MOE_Y_TOKEN_ORDER = 0x100 };
/* OR'd into the same regime: the DECODE partials' columns in partial-major
 * order (the plan then reports MOE_DTYPE_F32_PM).  With C = H/8 chunks of 8
 * columns and q = ceil(C/64), column c of chunk u = 64m + j (j < 64) is stored
 * at column 8(jq + m) + c mod 8: the chunks j, j+64, ... that form partial j
 * of the router's pinned logit sum lie side by side, so a reader that owns
 * partial j reads whole lines.  Needs C <= 64 or C a multiple of 64. */
enum { MOE_Y_PARTIAL_ORDER = 0x400 };
/* y dtypes: fp16, fp32 (decode slices), fp32 in partial-major column order;
 * bf16 where a call names it (moe_route_select, moe_quantize_fp8, moe_gemm_fp8,
 * moe_block_norm, moe_balance_loss). */
enum { MOE_DTYPE_F16 = 0, MOE_DTYPE_F32 = 1, MOE_DTYPE_F32_PM = 2, MOE_DTYPE_BF16 = 3 };
/* Expert blob formats: symmetric codes, or codes with a zero point per group
 * (lucashiago.com.br explainer, step 1: each block carries a scale and a zero
 * point).  MOE_W4_ZERO_POINT is OR'd into the regime of moe_expert_ffn_plan /
 * moe_expert_ffn_w4a16 / moe_pool_layer_args when the blobs are FMT_ZP. */
enum { MOE_FMT_SYM = 0, MOE_FMT_ZP = 1 };
/* Name of the FP8 blobs' format (moe_fp8_blob_layout) for programs that hold
 * layers of several formats; the _fmt calls refuse it (MOE_EINVAL). */
enum { MOE_FMT_FP8 = 2 };
enum { MOE_W4_ZERO_POINT = 0x200 };

/* Thread-local text of the last error on this thread ("" if none). */
const char *moe_last_error(void);

/*
 * Zero-fills ws_bytes bytes of a device workspace with a kernel on `stream`
 * (no hipMemsetAsync, so it may be recorded in a captured graph).  It is the
 * initial fill that moe_route_permute and moe_shared_ffn_f16 require, and the
 * way back after a call that did not run to completion (a failed launch, an
 * aborted graph replay): those calls keep an arrival ticket / arrival counters
 * at the start of their workspace, every completed call leaves them zero, and
 * a non-zero leftover would make the next call skip its final reduction.
 * Any address and size; MOE_EINVAL for a null ws with ws_bytes > 0.
 */
int moe_workspace_clear(void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------- expert blob */
/*
 * Canonical expert blob (Horizon RunMap "02 / A solução": compact weights
 * and FP16 scales in separate formats; lucashiago.com.br explainer step 1:
 * every block of weights carries its scale).  Six sections, each 256-byte
 * aligned:  gate_q[I][H/2], up_q[I][H/2], down_q[H][I/2]  (u8: element 2b in
 * the low nibble of byte b, element 2b+1 in the high nibble, stored as
 * u = q + 8 with q in [-7, 7]) then gate_s[I][H/g], up_s[I][H/g],
 * down_s[H][I/g] (fp16 scales, one per group of g along the input dim).
 * W = q * s.  offsets[6] get the section offsets, *total_bytes the blob size.
 * Host-only, no GPU needed.  MOE_EINVAL on bad sizes.
 */
int moe_blob_layout(int H, int I, int group, int64_t offsets[6], int64_t *total_bytes);

/*
 * Quantise n experts to canonical blobs on the device (symmetric group-wise
 * INT4; reading: s = fp16_rne(fp32(amax/7)), q = clamp(rne(fp32(w/s)), -7, 7),
 * q = 0 when s = 0).
 *   wg, wu: device fp32 [n][I][H]; wd: device fp32 [n][H][I] (row-major)
 *   blobs:  device, n consecutive blobs of total_bytes each (output)
 * Offline step (load time), not part of the per-token path.
 */
int moe_quantize_experts(const float *wg, const float *wu, const float *wd,
                         int n, int H, int I, int group, void *blobs, hipStream_t stream);

/*
 * Byte bijection from canonical blobs to the device layout the kernels read
 * (same size; never expands to fp16).  Applied once at load, to resident
 * weights and to the pinned source of the slot pool.
 *   src: device, n canonical blobs; dst: device, n blobs (must not overlap src)
 * Device layout: gate and up rows fused into 64-row blocks (32 gate rows then
 * the 32 up rows of the same intermediate indices), down in 64-row blocks;
 * inside a block, 32-element input chunks of all 64 rows are contiguous
 * (16 bytes per row: four dwords holding elements 0-7, 16-23, 8-15, 24-31,
 * each with element 2i at bits 4i and element 2i+1 at bits 16+4i, so that
 * a nibble pair converts in registers with one mask);
 * scales in [block][group][64 rows] order.
 */
int moe_prepack_experts(const void *src, int n, int H, int I, int group, void *dst,
                        hipStream_t stream);

/* Inverse of moe_prepack_experts (for inspection and tests). */
int moe_unpack_experts(const void *src, int n, int H, int I, int group, void *dst,
                       hipStream_t stream);

/*
 * Zero-point (asymmetric) INT4 blobs (lucashiago.com.br explainer, step 1:
 * each block of weights carries a scale and a zero point).  Canonical blob:
 * the six sections above at the same offsets, then gate_z[I][H/g],
 * up_z[I][H/g], down_z[H][I/g] (u8, one zero point z in [0, 15] per group),
 * each 256-byte aligned; a stored nibble u in [0, 15] means W = (u - z) * s.
 * (MOE_FMT_SYM is the case z = 8 with no zero-point sections.)
 * moe_blob_layout_fmt: offsets[0..8] (the last three 0 for MOE_FMT_SYM).
 * moe_quantize_experts_fmt with MOE_FMT_ZP quantises per group with the
 * reading lo = min(min w, 0), hi = max(max w, 0), s = fp16_rne((hi - lo)/15),
 * z = clamp(rne(-lo/s), 0, 15), u = clamp(rne(w/s) + z, 0, 15), quotients in
 * fp32; s = 0 gives z = u = 0.  moe_prepack_experts_fmt /
 * moe_unpack_experts_fmt: the device layout of moe_prepack_experts plus the
 * zero points in the scales' order (one byte each) after the scales.  The
 * expert kernels read such blobs when MOE_W4_ZERO_POINT is OR'd into the
 * regime.  MOE_EINVAL for an unknown fmt, else as the symmetric calls.
 */
int moe_blob_layout_fmt(int H, int I, int group, int fmt, int64_t offsets[9],
                        int64_t *total_bytes);
int moe_quantize_experts_fmt(const float *wg, const float *wu, const float *wd, int n, int H,
                             int I, int group, int fmt, void *blobs, hipStream_t stream);
int moe_prepack_experts_fmt(const void *src, int n, int H, int I, int group, int fmt, void *dst,
                            hipStream_t stream);
int moe_unpack_experts_fmt(const void *src, int n, int H, int I, int group, int fmt, void *dst,
                           hipStream_t stream);

/*
 * The same bijection on the host, one blob (src and dst host memory of the
 * canonical blob size, not overlapping): for a source that lives in host
 * memory, such as the pinned INT4 source of the slot pool, so that loading it
 * needs no device round trip.  Bytes identical to moe_prepack_experts_fmt /
 * moe_unpack_experts_fmt.  No GPU needed.  MOE_EINVAL on bad arguments.
 */
int moe_prepack_expert_host(const void *src, int H, int I, int group, int fmt, void *dst);
int moe_unpack_expert_host(const void *src, int H, int I, int group, int fmt, void *dst);

/* ------------------------------------------------------------ router */
/*
 * Router softmax + top-k (Horizon RunMap "03 / Arquitetura": the router
 * selects the experts of each token; routing stays outside INT4, "08").
 *   x_f16:        device fp16 [T][H] activations
 *   w_router_f16: device fp16 [E][H]
 *   logit_bias:   device fp32 [E] added to every logit after the dot product,
 *                 or NULL
 *   flags:        MOE_RENORM renormalises the k weights to sum to one
 *   topk_idx:     device int32 [T][k] (output), experts by (logit desc,
 *                 index asc) -- ties go to the lower expert index
 *   topk_w:       device fp32 [T][k] (output), softmax over all E logits at
 *                 the chosen experts
 *   ws:           device scratch of moe_route_workspace_bytes(T, E) bytes
 *                 (0 for T <= 8, where ws may be NULL; above that it holds the
 *                 T x E fp32 logits between the logit and top-k launches;
 *                 contents need no initialisation); MOE_ENOMEM if too small
 * Logits are fp32 in a fixed summation order (chunks of 8 elements of H go
 * to partial (chunk mod 64) in increasing order, partials combined by an xor
 * butterfly 32,16,8,4,2,1), so the indices are reproducible bit for bit.
 * T = 0 is a no-op.
 */
size_t moe_route_workspace_bytes(int T, int E);
int moe_route(const void *x_f16, const void *w_router_f16, const float *logit_bias,
              int T, int H, int E, int k, unsigned flags,
              int32_t *topk_idx, float *topk_w, void *ws, size_t ws_bytes,
              hipStream_t stream);

/* ------------------------------------------------------- permutation */
/*
 * Token-to-expert grouping (the pages' grouped executor computes experts in
 * groups, Horizon RunMap "04 / Resultados").  Stable counting sort of the
 * flat index f = t*k + j by expert topk_idx[f]:
 *   counts   device int32 [E]     tokens routed to each expert
 *   offsets  device int32 [E+1]   exclusive scan of counts, offsets[E] = T*k
 *   perm     device int32 [T*k]   sorted position -> f (f ascending per expert)
 *   inv_perm device int32 [T*k]   f -> sorted position
 * ws: device scratch of at least moe_permute_workspace_bytes(T, k, E) bytes
 * (contents need no initialisation).  Bit-exact: one correct answer.
 */
size_t moe_permute_workspace_bytes(int T, int k, int E);
int moe_permute(const int32_t *topk_idx, int T, int k, int E,
                int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *inv_perm,
                void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * moe_route followed by moe_permute, with the same arguments and results
 * (same passages and readings).  For small T (T <= 5 with E <= 128, T <= 4
 * with E > 128, where one selecting workgroup still beats two launches) both
 * run in one launch: the logits are spread over many workgroups, and the
 * workgroup that finishes last (an atomic ticket in ws; no workgroup ever
 * waits for another) does the top-k, the softmax and the stable sort -- the
 * decode path's one launch instead of two.  For larger T it runs moe_route's
 * launches (logits into ws, then top-k) followed by moe_permute's, on the
 * same ws.
 * ws: device scratch of moe_route_permute_workspace_bytes(T, k, E) bytes.  It
 * must be zero-filled before its first use by this function; every completed
 * call leaves it reusable (the ticket, its first 256 bytes, back at zero),
 * for any T.  Calls that share one workspace must not run concurrently.
 */
size_t moe_route_permute_workspace_bytes(int T, int k, int E);
int moe_route_permute(const void *x_f16, const void *w_router_f16, const float *logit_bias,
                      int T, int H, int E, int k, unsigned flags,
                      int32_t *topk_idx, float *topk_w, int32_t *counts, int32_t *offsets,
                      int32_t *perm, int32_t *inv_perm, void *ws, size_t ws_bytes,
                      hipStream_t stream);

/*
 * moe_route_permute without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  Same arguments (minus ws), results and
 * errors as moe_route_permute; it calls no hipMalloc/hipFree and no
 * allocating routine.  Its workspace is a 16 MiB array inside the library, one
 * per GPU, held until the process ends; on the first call on a device its
 * ticket is cleared by a kernel on `stream`, and every completed call leaves
 * it clear again.  Shapes whose workspace (moe_route_permute_workspace_bytes)
 * exceeds 16 MiB are rejected with MOE_ENOMEM before anything is launched
 * (T = 4096 tokens with E = 512 experts and k = 10 need 8.7 MB; the
 * workspace grows as 4*T*E bytes).  Every call on one GPU shares that
 * array: calls that overlap in time on one GPU (different streams, or
 * threads) race and must not be made.
 */
int moe_route_permute_noalloc(const void *x_f16, const void *w_router_f16,
                              const float *logit_bias, int T, int H, int E, int k, unsigned flags,
                              int32_t *topk_idx, float *topk_w, int32_t *counts, int32_t *offsets,
                              int32_t *perm, int32_t *inv_perm, hipStream_t stream);

/* ------------------------------------------------ routed expert FFN */
/*
 * What moe_expert_ffn_w4a16 will do for a shape: the resolved regime, the
 * dtype and number of slices of y, and the workspace it needs.  Host-only.
 * AUTO picks DECODE for T <= 4 tokens, SMALL for T <= 32, else BATCHED.
 *   DECODE : one launch, rows of an expert one after another on the vector
 *            ALUs.  y is fp32 [slices][T*k][H], partial sums over
 *            intermediate slices of 32 (slices = I/32); moe_combine adds them.
 *   SMALL  : T <= 32 (Horizon RunMap "10 / Próximas perguntas": concurrent
 *            use).  Each expert's weights are streamed once and its <= T rows
 *            multiplied on the matrix cores; gate/up then down, h in ws.
 *            T > 32 is MOE_EUNSUPPORTED.  y is fp16 [1][T*k][H].
 *   BATCHED: tiled grouped GEMM, any T.  y is fp16 [1][T*k][H].
 * regime may carry MOE_Y_TOKEN_ORDER and MOE_Y_PARTIAL_ORDER (DECODE only:
 * MOE_EUNSUPPORTED when the resolved regime is another; with the second, y_dtype
 * is MOE_DTYPE_F32_PM) and MOE_W4_ZERO_POINT (any regime: the blobs are
 * MOE_FMT_ZP); resolved_regime is returned without them.
 */
int moe_expert_ffn_plan(int T, int H, int I, int E, int k, int group, int regime,
                        int *resolved_regime, int *y_dtype, int *y_slices,
                        size_t *ws_bytes);

/*
 * Routed-expert SwiGLU FFN computed directly from INT4 weights
 * (Horizon RunMap "03 / Arquitetura" and "08": the kernel reads compact
 * weights and FP16 scales, converts what it needs during the computation,
 * uses FP16 activations and FP32 accumulation, and never keeps an expanded
 * expert).  For each sorted row p of expert e and token t = perm[p] / k:
 *   h = silu(Wg[e] x_t) * (Wu[e] x_t),   y_p = Wd[e] h,   W = q * s.
 *   x_f16          device fp16 [T][H]; 16-byte aligned
 *   perm, offsets  device, from moe_permute
 *   d_expert_blobs device array of E device pointers to prepacked blobs
 *                  (moe_prepack_experts); an entry may be NULL only for an
 *                  expert no token routes to, except in the DECODE regime,
 *                  where a routed expert with a NULL entry is skipped (its y
 *                  rows are left unwritten for another launch to fill)
 *   y              device output, layout from moe_expert_ffn_plan, 16-byte
 *                  aligned; y_dtype and y_slices must equal the plan's
 *                  (MOE_EINVAL otherwise).
 *                  Row p holds sorted row p; with MOE_Y_TOKEN_ORDER in regime
 *                  (DECODE only) the result of sorted row p goes to row
 *                  perm[p] = t*k + j instead, so that moe_combine needs no
 *                  inv_perm (one dependent memory round trip less); with
 *                  MOE_Y_PARTIAL_ORDER each row's columns are stored in
 *                  partial-major order (MOE_DTYPE_F32_PM)
 *   ws             device scratch of the plan's size (may be NULL if 0)
 * Rounding: DECODE converts h to fp16 before the down projection; SMALL and
 * BATCHED convert the weights to fp16(q * s) and store h and y as fp16.
 * Everything else accumulates in fp32.
 */
int moe_expert_ffn_w4a16(const void *x_f16, const int32_t *perm, const int32_t *offsets,
                         const void *const *d_expert_blobs,
                         int T, int H, int I, int E, int k, int group, int regime,
                         void *y, int y_dtype, int y_slices,
                         void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------ shared FP16 expert */
/*
 * Separate FP16 non-routed expert (Horizon RunMap "03": parts outside the
 * routed experts stay FP16).  SwiGLU FFN applied to every token:
 *   s_t = Wd (silu(Wg x_t) * (Wu x_t)),
 *   wg, wu: device fp16 [Is][H];  wd: device fp16 [H][Is]  (row-major)
 *   out_f32: device fp32 [T][H]
 *   ws:      device scratch of moe_shared_ffn_workspace_bytes(T, H, Is) bytes,
 *            zero-filled by the caller before its first use.  Its first 2 KB
 *            hold arrival counters of the split-K reduction; every call
 *            leaves them zero again, so one zero-fill serves any number of
 *            calls (and graph replays) with any T.  Calls that share a
 *            workspace must not overlap.
 * h is rounded to fp16 between the projections; fp32 accumulation.  The
 * order of the fp32 additions depends on T, H and Is only, so repeated calls
 * give identical bits.
 */
size_t moe_shared_ffn_workspace_bytes(int T, int H, int Is);
int moe_shared_ffn_f16(const void *x_f16, const void *wg, const void *wu, const void *wd,
                       int T, int H, int Is, float *out_f32,
                       void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------ combine */
/*
 * Router-weighted combine (Horizon RunMap "03": results go back to the rest
 * of the model).  For each token t and column c:
 *   out[t,c] = fp16_rne( r + sum_j w[t,j] * Y(inv_perm[t*k+j], c) + s[t,c] )
 * where Y(p,c) is y[p,c] (y_dtype F16, y_slices 1) or the sum over slices of
 * y[slice][p][c] (F32; the slices summed in two contiguous halves, each in
 * slice order, then the halves added; F32_PM: the same with column c read
 * from its partial-major position), r = residual[t,c] or 0, s the
 * shared-expert output or 0.  fp32 sum in the order: experts j = 0..k-1
 * (each the slice sum), shared, residual; one final rounding.
 *   y            device, from moe_expert_ffn_w4a16; 16-byte aligned
 *   inv_perm     device int32 [T*k], or NULL when y is in token order
 *                (MOE_Y_TOKEN_ORDER): then Y(t*k+j, c) is read directly
 *   topk_w       device fp32 [T][k]
 *   shared_f32   device fp32 [T][H] or NULL
 *   residual_f16 device fp16 [T][H] or NULL (may alias out_f16)
 *   out_f16      device fp16 [T][H]
 * Errors: MOE_EINVAL for bad sizes or dtype (k outside 1..16, F16 y with
 * more than one slice, F32_PM with an H that has no partial-major order), a
 * null y/topk_w/out pointer or a misaligned y; MOE_EUNSUPPORTED when H is
 * not a multiple of 8.
 */
int moe_combine(const void *y, int y_dtype, int y_slices, const int32_t *inv_perm,
                const float *topk_w, const float *shared_f32, const void *residual_f16,
                int T, int H, int k, void *out_f16, hipStream_t stream);

/*
 * Combine with a gated shared expert.  The pages run a second model family
 * with 60 routed experts per layer and a top-4 executor (Horizon RunMap
 * technical preview, residency results table, top4-fused-v1 rows) without
 * printing its layer; in that family the shared expert's output is scaled per
 * token by a sigmoid of one more linear function of the token (a reading; no
 * bias term).  Same as moe_combine except that the shared term is
 *   G_t * s[t,c],   G_t = 1 / (1 + exp(-sum_c x[t,c] * wsg[c])),
 * the dot taken in fp32 (any order; G_t is not a discrete decision).
 *   shared_f32         device fp32 [T][H], required
 *   x_f16              device fp16 [T][H], the layer input; 16-byte aligned
 *   shared_gate_w_f16  device fp16 [H]; 16-byte aligned
 * Errors: MOE_EINVAL for a null shared/x/gate pointer or misalignment, else
 * as moe_combine.
 */
int moe_combine_gated(const void *y, int y_dtype, int y_slices, const int32_t *inv_perm,
                      const float *topk_w, const float *shared_f32, const void *x_f16,
                      const void *shared_gate_w_f16, const void *residual_f16, int T, int H,
                      int k, void *out_f16, hipStream_t stream);

/*
 * Combine of one layer fused with route + permute of the next (Horizon
 * RunMap "03 / Arquitetura": the experts' results return to the model, whose
 * next layer's router then selects its experts; the pages run 16 such layers
 * per token).  Exactly the two calls it stands for, bit for bit:
 *   moe_combine (shared_gate_w_f16 NULL) or moe_combine_gated (non-NULL:
 *     then shared_f32 and x_f16, the layer's input, are required) with y,
 *     y_dtype, y_slices, inv_perm, topk_w, shared_f32, residual_f16, T, H, k,
 *     writing out_f16;
 *   then moe_route_permute(out_f16, w_router_f16, logit_bias, T, H, E, k_next,
 *     flags, topk_idx, topk_w_next, counts, offsets, perm, inv_perm_next).
 * One launch when T = 1, E <= 64 and y holds fp32 slices (y_slices > 1, the
 * decode layout; with MOE_DTYPE_F32_PM every block of that launch reads whole
 * lines); otherwise the two calls run in turn on `stream`.
 *   ws  device workspace of moe_combine_route_permute_workspace_bytes(T,
 *       k_next, E) bytes, zero-filled before the first call
 *       (moe_workspace_clear).  The fused launch leaves its first 256 bytes
 *       alone and passes the next layer's logit partials from block to block
 *       through tagged words after them (the selecting block polls them; no
 *       other block waits), with a call counter at the end; so the same
 *       workspace may also serve moe_route_permute, whose ticket lives in the
 *       first 256 bytes.
 * The layer's routing arrays (topk_w, inv_perm) and the next layer's
 * (topk_w_next, inv_perm_next) may be the same arrays: every read of the
 * former precedes every write of the latter.  out_f16 may alias residual_f16
 * but not x_f16.  Errors: those of the two calls, checked before any launch;
 * MOE_ENOMEM for a short workspace.
 */
size_t moe_combine_route_permute_workspace_bytes(int T, int k_next, int E);
int moe_combine_route_permute(const void *y, int y_dtype, int y_slices, const int32_t *inv_perm,
                              const float *topk_w, const float *shared_f32, const void *x_f16,
                              const void *shared_gate_w_f16, const void *residual_f16, int T,
                              int H, int k, void *out_f16, const void *w_router_f16,
                              const float *logit_bias, int E, int k_next, unsigned flags,
                              int32_t *topk_idx, float *topk_w_next, int32_t *counts,
                              int32_t *offsets, int32_t *perm, int32_t *inv_perm_next, void *ws,
                              size_t ws_bytes, hipStream_t stream);

/*
 * The same two stacked decode layers split differently: the combine of
 * layer l and only the next layer's logit partials in one launch, then the
 * next layer's routing done inside its expert FFN.  Every workgroup of the
 * FFN folds the partials in the pinned order and selects for itself, so no
 * workgroup waits for another and the combine's launch ends once its
 * partials are stored.  Together the two calls give, bit for bit, what
 * moe_combine_route_permute followed by moe_expert_ffn_w4a16 give (the same
 * out_f16, routing arrays and y).  For one decode token of at most 64 experts
 * (T = 1, E <= 64, y of the decode regime: MOE_DTYPE_F32 or MOE_DTYPE_F32_PM
 * with y_slices > 1); other shapes are MOE_EUNSUPPORTED (use the calls above).
 *
 * moe_combine_route_partials: arguments as moe_combine_route_permute up to
 * logit_bias-less w_router_f16 and E; writes out_f16 and
 *   logit_partials  device fp32 [64][64] (moe_logit_partials_bytes()):
 *                   partial j of expert e's logit at j * 64 + e, partial j
 *                   summing the 8-column chunks j, j + 64, ... of out_f16 in
 *                   the pinned order (Horizon RunMap "08": routing in FP32
 *                   with explicit roundings); rows j >= min(64, H / 8) are not
 *                   written and count as zero.
 * moe_expert_ffn_w4a16_routed: x_f16 (the combine's out_f16), the partials,
 * logit_bias (may be NULL), E, k, flags as moe_route; writes the routing
 * arrays of moe_route_permute (topk_idx, topk_w, counts, offsets, perm,
 * inv_perm) and y as moe_expert_ffn_w4a16 in the DECODE regime (regime may
 * carry MOE_Y_TOKEN_ORDER, MOE_Y_PARTIAL_ORDER and MOE_W4_ZERO_POINT;
 * d_expert_blobs must hold every expert).  Errors: MOE_EINVAL / ENOMEM /
 * EUNSUPPORTED as the calls they replace, checked before any launch.
 * moe_logit_partials: the same partials straight from an fp16 input row
 * that no combine forms (the first layer of a stack): x_f16 device fp16 [H]
 * (T = 1), w_router_f16 device fp16 [E][H] (both 16-byte aligned), into
 * logit_partials as above; routing from them equals moe_route_permute of
 * x_f16 bit for bit.  One launch of min(64, H / 8) one-wave workgroups.
 * Errors: MOE_EINVAL (shape, null, alignment), MOE_EUNSUPPORTED (T != 1,
 * E > 64, H not instantiated), before any launch.
 */
size_t moe_logit_partials_bytes(void);
int moe_logit_partials(const void *x_f16, const void *w_router_f16, int T, int H, int E,
                       float *logit_partials, hipStream_t stream);
int moe_combine_route_partials(const void *y, int y_dtype, int y_slices, const int32_t *inv_perm,
                               const float *topk_w, const float *shared_f32, const void *x_f16,
                               const void *shared_gate_w_f16, const void *residual_f16, int T,
                               int H, int k, void *out_f16, const void *w_router_f16, int E,
                               float *logit_partials, hipStream_t stream);
int moe_expert_ffn_w4a16_routed(const void *x_f16, const float *logit_partials,
                                const float *logit_bias, int E, int k, unsigned flags,
                                int32_t *topk_idx, float *topk_w, int32_t *counts,
                                int32_t *offsets, int32_t *perm, int32_t *inv_perm,
                                const void *const *d_expert_blobs, int T, int H, int I,
                                int group, int regime, void *y, int y_dtype, int y_slices,
                                hipStream_t stream);

/* ------------------------------------------- routing by scores and groups */
/*
 * Router logits alone: the logits that moe_route selects from (same summation
 * order, same bits), for a selection the caller runs itself or with
 * moe_route_select.
 *   x_f16 device fp16 [T][H], w_router_f16 device fp16 [E][H] (16-byte
 *   aligned), logit_bias device fp32 [E] or NULL; logits device fp32 [T][E].
 * H in {256, 512, 1024, 2048}, E <= 1024, T <= 2^27 - 8 (MOE_EUNSUPPORTED).
 * T = 0: no-op.
 */
int moe_router_logits(const void *x_f16, const void *w_router_f16, const float *logit_bias, int T,
                      int H, int E, float *logits, hipStream_t stream);

/*
 * Expert selection from logits in hand, in the forms of current sparse
 * models.  With l the logits of a token:
 *   s_e = softmax(l)_e (MOE_SCORE_SOFTMAX) or 1 / (1 + exp(-l_e))
 *         (MOE_SCORE_SIGMOID);
 *   c_e = s_e + select_bias[e]  -- a balancing bias decides, it does not weigh;
 *   the experts are n_group equal runs of E / n_group; a group counts by its
 *   largest c, or with MOE_GROUP_TOP2 by the sum of its two largest; only the
 *   topk_group groups that count most (ties: lower group) can be chosen from;
 *   topk_idx: the k largest c in descending order (ties: lower expert);
 *   topk_w:   scale * s at those experts, with MOE_RENORM divided by the sum
 *             of the k chosen s (all zero when that sum is zero).
 * A logit of -inf or NaN masks its expert: s = 0, and it ranks behind every
 * other expert of the kept groups (by index) and does not count for its
 * group; a row that is masked throughout gives the lowest experts of the
 * lowest groups with weight 0.  A logit of +inf counts as the largest finite
 * value, a choice that is NaN ranks as masked.  Scores and choices are formed
 * in fp64; topk_w is rounded once.
 *   logits      device [T] rows of E values of logits_dtype (MOE_DTYPE_F32,
 *               F16 or BF16), ld elements apart (ld >= E), element-aligned
 *   select_bias device fp32 [E] or NULL
 *   topk_idx    device int32 [T][k];  topk_w device fp32 [T][k]
 * Errors: MOE_EINVAL for bad sizes (n_group must divide E; the kept groups
 * must hold k experts; ld < E), an unknown dtype, score or flag, a scale that
 * is not finite, null or misaligned pointers; MOE_EUNSUPPORTED for E > 1024,
 * k > 16, more than 64 groups or T > 2^25.  T = 0: no-op (the permute form
 * then gives empty groups).
 * The permute form also writes moe_permute's outputs of topk_idx, in the same
 * launch for one token (and up to 16 with T * E <= 8192), in one more up to
 * 8192 tokens of 768 experts, else by moe_permute's launches.
 *   ws  device scratch of moe_route_select_workspace_bytes(T, k, E) bytes (may
 *       be 0; no initialisation needed), 16-byte aligned; MOE_ENOMEM if too
 *       small.  Calls that share it must not overlap.
 */
int moe_route_select(const void *logits, int logits_dtype, int64_t ld, const float *select_bias,
                     int T, int E, int k, int score, int n_group, int topk_group, unsigned flags,
                     float scale, int32_t *topk_idx, float *topk_w, hipStream_t stream);
size_t moe_route_select_workspace_bytes(int T, int k, int E);
int moe_route_select_permute(const void *logits, int logits_dtype, int64_t ld,
                             const float *select_bias, int T, int E, int k, int score, int n_group,
                             int topk_group, unsigned flags, float scale, int32_t *topk_idx,
                             float *topk_w, int32_t *counts, int32_t *offsets, int32_t *perm,
                             int32_t *inv_perm, void *ws, size_t ws_bytes, hipStream_t stream);

/* --------------------------------------------- FP8 with block scales (W8A8) */
/*
 * e4m3 (OCP: 1 sign, 4 exponent, 3 mantissa bits, largest value 448) with one
 * fp32 scale per block: x is about q * s.
 * moe_quantize_fp8: blocks of block_rows x 128 (block_rows 1: activations,
 * one scale per row and 128 columns; 128: weights), the last ones partial.
 *   a = max |x| of the block; s = a / 448 in fp32, at least 2^-126 (0 when
 *   a = 0); with MOE_SCALE_POW2 the smallest power of two not below that (then
 *   x / s is exact); q = e4m3(x / s), nearest even (0 when s = 0).
 *   x       device [rows] of cols values of dtype (F16, BF16, F32), ldx
 *           elements apart, element-aligned (fastest 16-byte aligned)
 *   q       device e4m3 [rows], ldq bytes apart (fastest 8-byte aligned)
 *   scales  device fp32 [ceil(rows / block_rows)][ceil(cols / 128)]
 * A block that holds a NaN or an infinity gives codes or a scale that make
 * every product with it NaN or infinite.  q and scales must not overlap x.
 * Errors: MOE_EINVAL for bad sizes, dtype, block_rows or flags, null or
 * misaligned pointers; MOE_EUNSUPPORTED for cols > 2^30 or more than
 * 2^36 row blocks; rows = 0: no-op.
 */
int moe_quantize_fp8(const void *x, int dtype, int64_t ldx, int64_t rows, int cols, int block_rows,
                     unsigned flags, void *q, int64_t ldq, float *scales, hipStream_t stream);

/*
 * Dense product of two such matrices, y = x w^T:
 *   y[m][n] = sum_b xs[m][b] * ws[n/128][b] * sum_{j in block b} xq[m][j] wq[n][j]
 * a block's sum formed on the matrix cores, scaled once, the blocks accumulated
 * in fp32 in a fixed order, rounded once to out_dtype.  fp32 outputs have the
 * accuracy of fp32 sums.  16-bit outputs of many rows take the FP8 matrix
 * instruction, which adds runs of eight neighbouring products and drops there
 * what lies 13 bits below the run's largest (1.4e-5 relative on random data,
 * below the output's own rounding; at worst 7 * 2^-13 of the sum of |products|,
 * which exceeds that rounding where products cancel).  With MOE_ACC_F32 OR'd
 * into out_dtype 16-bit outputs have the accuracy of fp32 sums at every size,
 * so that a row's does not depend on how many rows come with it, at half the
 * instruction's rate.
 *   xq  device e4m3 [M], ldx bytes apart;  x_scales device fp32 [M][ceil(K/128)]
 *   wq  device e4m3 [N], ldw bytes apart;  w_scales [ceil(N/128)][ceil(K/128)]
 *   out device [M] rows of N values (F16, BF16 or F32), ldo elements apart
 * M and N up to 2^31 - 256 and 2^23 tiles of 256 x 256 (M <= 2097120 and N <=
 * 2^28 where ldw >= 2^22); K, ldx and ldw multiples of 16, K <= 16384
 * (MOE_EUNSUPPORTED otherwise); xq and wq 16-byte aligned (MOE_EINVAL).  out
 * must not overlap the inputs.  M = 0: no-op.  No workspace.
 */
int moe_gemm_fp8(const void *xq, int64_t ldx, const float *x_scales, const void *wq, int64_t ldw,
                 const float *w_scales, int M, int N, int K, void *out, int out_dtype, int64_t ldo,
                 hipStream_t stream);

/*
 * FP8 expert blob: six sections, each 256-byte aligned: gate_q[I][H],
 * up_q[I][H], down_q[H][I] (e4m3, row-major) then gate_s, up_s
 * [ceil(I/128)][ceil(H/128)] and down_s[ceil(H/128)][ceil(I/128)] (fp32, one
 * per 128 x 128 block) -- moe_quantize_fp8 with block_rows = 128 writes such
 * sections.  The kernels read this layout as it is.  Host-only.  H and I up to
 * 2^30 (MOE_EUNSUPPORTED).
 */
int moe_fp8_blob_layout(int H, int I, int64_t offsets[6], int64_t *total_bytes);

/*
 * Routed SwiGLU experts from FP8 blobs.  For each sorted row p of expert e and
 * token t = perm[p] / k:
 *   (xq, xs) = quantised x_t,  g = Wg[e] x, u = Wu[e] x (products as above),
 *   h = silu(g) * u in fp32,   (hq, hs) = quantised h,   y_p = Wd[e] h -> fp16
 * the activations quantised per row and 128 columns with power-of-two scales
 * (MOE_SCALE_POW2).
 *   x_f16, perm, offsets, d_expert_blobs as moe_expert_ffn_w4a16 (a NULL entry
 *   leaves that expert's rows of y unwritten); blobs in the layout above,
 *   16-byte aligned
 *   y_f16  device fp16 [T*k][H], row p holds sorted row p (moe_combine with
 *          MOE_DTYPE_F16, one slice)
 *   ws     device scratch of the plan's size, 16-byte aligned, no
 *          initialisation; calls that share it must not overlap
 * A token with a NaN or an infinity has no finite value in its rows.
 * Rows behind offsets[E] are left as they were.  Regimes: DECODE (T <= 128 and
 * min(T, 16) * ceil(max(H, I) / 128) <= 600, else MOE_EUNSUPPORTED: two
 * launches over the weights' stream, activations quantised inside them) and
 * BATCHED (T * ceil(H / 128) up to 2^28 - 32, and at most 2^23 - 8 tiles a
 * launch, rounded up: (T k / rows + min(E, T k)) * max(I / 128, H / 256) with
 * tiles of 64 to 192 rows; MOE_EUNSUPPORTED beyond, also by the plan); AUTO takes DECODE where it can
 * up to T * k = 64, and up to 192 while T * k * ceil(H / 128) <= 1024.  The sums of DECODE and of BATCHED's gate and up have fp32
 * accuracy; BATCHED's down is a 16-bit output as above, and MOE_ACC_F32 OR'd into
 * the regime (the resolved one keeps it) gives its sums fp32 accuracy too.  H and I multiples of
 * 64, at most 8192; E <= 1024; k <= 16 (MOE_EUNSUPPORTED).  x, y and ws 16-byte
 * aligned (MOE_EINVAL).  T = 0: no-op.
 */
int moe_expert_ffn_w8a8_plan(int T, int H, int I, int E, int k, int regime, int *resolved_regime,
                             size_t *ws_bytes);
int moe_expert_ffn_w8a8(const void *x_f16, const int32_t *perm, const int32_t *offsets,
                        const void *const *d_expert_blobs, int T, int H, int I, int E, int k,
                        int regime, void *y_f16, void *ws, size_t ws_bytes, hipStream_t stream);

/* -------------------------------------------- around the block: norms */
/*
 * The end of one block and the start of the next, for each of T rows of H:
 *   u = post(y) with MOE_NORM_POST, else y
 *   r = residual + scale * gate * u          (out, rounded once)
 *   n = pre(r), of the unrounded r           (n, rounded once)
 * with the norms of `kind`, over the H columns,
 *   RMS:   x / sqrt(mean(x^2) + eps) * w + b
 *   LAYER: (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * w + b
 * in fp32; with MOE_NORM_UNIT_OFFSET 1 + w stands for w.
 *   y, residual  device [T] rows of `dtype` (F16, BF16 or F32), ldy and ldr
 *                elements apart, element-aligned (fastest 16-byte aligned);
 *                either may be NULL (zeros), not both; gate and post norm need y
 *   gate         device [H] of dtype for all tokens (ldg = 0), or [T] rows ldg
 *                apart; NULL: ones
 *   post_w, post_b, pre_w, pre_b  device [H] of w_dtype (dtype or F32), each may
 *                be NULL (w: ones, whatever the flags; b: zeros); post ones need
 *                MOE_NORM_POST, pre ones need n
 *   out, n       device [T] rows of dtype, ldo and ldn apart; either may be NULL,
 *                not both.  They may be y, residual or gate rows themselves (the
 *                same address and stride); no other overlap.
 * Squares are summed in fp32: rows with values beyond 2^60 overflow there.  A row
 * that holds a NaN or an infinity affects no other row.  H <= 8192
 * (MOE_EUNSUPPORTED).  T = 0: no-op.  No workspace.
 */
int moe_block_norm(const void *y, int64_t ldy, const void *residual, int64_t ldr, const void *gate,
                   int64_t ldg, float scale, const void *post_w, const void *post_b,
                   const void *pre_w, const void *pre_b, int dtype, int w_dtype, int kind,
                   unsigned flags, float eps, int T, int H, void *out, int64_t ldo, void *n,
                   int64_t ldn, hipStream_t stream);

/*
 * Gradients of moe_block_norm from those of out and n (dout, dn: either may be
 * NULL, not both; without dn there is no pre norm) and the forward call's inputs.
 * A gradient of rows is laid out as the rows: dy as y (ldy), dresidual as
 * residual (ldr), dgate as gate (ldg); dout and dn lie ldo and ldn apart.
 *   dy, dresidual  device rows of dtype, or NULL
 *   dgate          ldg = 0: device fp32 [H], the sum over the tokens; else rows of
 *                  dtype; or NULL
 *   dpost_w, dpost_b, dpre_w, dpre_b  device fp32 [H], sums over the tokens, or
 *                  NULL; their order of addition depends on T and H only
 * Everything is formed in fp32 and rounded once.  dy and dresidual may be dout or
 * dn rows themselves (same address and stride), or y, residual, gate.
 *   ws  device scratch of moe_block_norm_backward_workspace_bytes(T, H) bytes
 *       where a sum over the tokens is asked for, 16-byte aligned, no
 *       initialisation; calls that share it must not overlap
 * T = 0: the sums are set to zero.
 */
size_t moe_block_norm_backward_workspace_bytes(int T, int H);
int moe_block_norm_backward(const void *dout, int64_t ldo, const void *dn, int64_t ldn,
                            const void *y, int64_t ldy, const void *residual, int64_t ldr,
                            const void *gate, int64_t ldg, float scale, const void *post_w,
                            const void *post_b, const void *pre_w, int dtype, int w_dtype, int kind,
                            unsigned flags, float eps, int T, int H, void *dy, void *dresidual,
                            void *dgate, float *dpost_w, float *dpost_b, float *dpre_w,
                            float *dpre_b, void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------ around the block: products */
/*
 * fp16 product with its epilogue:
 *   z = x w^T + bias,   out = residual + act(z)
 * summed in fp32; bias, activation and residual are applied before the one
 * rounding to out_dtype.
 *   x_f16     device fp16 [M] rows of K values, ldx apart; 16-byte aligned
 *   w_f16     device fp16 [N] rows of K values, ldw apart; 16-byte aligned
 *   bias      device fp32 [N] or NULL;  act: MOE_ACT_*
 *   residual  device [M] rows of N values of out_dtype, ldr apart, or NULL; may be
 *             out itself
 *   out       device [M] rows of N values of out_dtype (F16 or F32), ldo apart
 *   z_f16     device fp16 [M] rows of N values, ldz apart, or NULL: z rounded, as
 *             moe_linear_f16_backward takes it
 *   ws        device scratch of moe_linear_f16_workspace_bytes(M, N, K) bytes (may
 *             be 0), 16-byte aligned, no initialisation; calls that share it must
 *             not overlap
 * The order of the fp32 additions depends on M, N and K only.  K, ldx and ldw are
 * multiples of 8, rows lie at most 2^22 elements apart, M and N are at most 2^30 and
 * small enough for a launch (at most 2^22 - 8 tiles of 256 x 256); else
 * MOE_EUNSUPPORTED.  M = 0: no-op.
 */
size_t moe_linear_f16_workspace_bytes(int M, int N, int K);
int moe_linear_f16(const void *x_f16, int64_t ldx, const void *w_f16, int64_t ldw,
                   const float *bias, int act, const void *residual, int64_t ldr, int M, int N,
                   int K, void *out, int out_dtype, int64_t ldo, void *z_f16, int64_t ldz, void *ws,
                   size_t ws_bytes, hipStream_t stream);

/*
 * Gradients of that product from dy, the gradient of out (which is also the
 * residual's):
 *   dz = dy * act'(z),   dx = dz w,   dw = dz^T x,   dbias = sum over rows of dz
 *   dy_f16  device fp16 [M] rows of N values, lddy apart
 *   z_f16   as the forward call wrote it (an infinity: beyond fp16, with the
 *           derivative's limit); not read with MOE_ACT_NONE
 *   x_f16, w_f16  as in the forward call (x is read for dw only, w for dx only)
 *   dx      device [M] rows of K values of out_dtype, lddx apart, or NULL
 *   dw      device [N] rows of K values of out_dtype, lddw apart, or NULL
 *   dbias   device fp32 [N] or NULL, from the unrounded dz
 *   ws      device scratch of moe_linear_f16_backward_workspace_bytes(M, N, K)
 *           bytes, as above
 * dz enters the products as it is with MOE_ACT_NONE and RELU, else as the sum of two
 * fp16 (off by 2^-21 of it, or 2^-25), at every size; so the products take twice the
 * operations.  With MOE_DZ_F16 OR'd into out_dtype it is rounded to one: half the
 * time, and 1.4 times the error in dx and dw (dbias is not affected).  out_dtype F32
 * is for MOE_ACT_NONE only (MOE_EUNSUPPORTED), and bits of out_dtype besides are refused.
 * Gradients that would leave fp16's range belong scaled by the caller.  Limits as above,
 * for the products of dx and dw, whichever is asked for, N at most 2^22, and M at most
 * 2^29 where dz is two fp16 (MOE_EUNSUPPORTED); lddy, ldz, lddx and lddw are free.
 * M = 0: dw and dbias are set to zero.
 */
size_t moe_linear_f16_backward_workspace_bytes(int M, int N, int K);
int moe_linear_f16_backward(const void *dy_f16, int64_t lddy, const void *z_f16, int64_t ldz,
                            int act, const void *x_f16, int64_t ldx, const void *w_f16, int64_t ldw,
                            int M, int N, int K, void *dx, int64_t lddx, void *dw, int64_t lddw,
                            int out_dtype, float *dbias, void *ws, size_t ws_bytes,
                            hipStream_t stream);

/* ------------------------------------------------- balance of the router */
/*
 * Per-expert counts, mean probabilities, balance loss and z loss of router logits,
 * and the logits' gradient.  Over the n tokens that token_mask does not mask, with
 * p the token's scores (MOE_SCORE_*) divided by their sum:
 *   counts[e] = choices of e in topk_idx,   f_e = counts[e] / sum of counts
 *   mean_prob[e] = 1/n sum_t p[t][e]
 *   losses[0] = coef * E * sum_e f_e mean_prob[e]
 *   losses[1] = z_coef / n * sum_t logsumexp(l_t)^2
 *   dlogits = *d_loss * d(losses[0] + losses[1]) / dlogits, the counts constant;
 *             zero for masked tokens
 * A logit of -inf or NaN masks its expert (p = 0, gradient 0), +inf counts as the
 * largest finite value, a token masked throughout has p = 0 and no z loss.
 *   logits      device [T] rows of E values of logits_dtype (F32, F16, BF16), ld
 *               apart, element-aligned
 *   topk_idx    device int32 [T][k], from moe_route or moe_route_select (an index
 *               outside [0, E) does not count), or NULL: counts is an input, such
 *               as moe_route_select_permute's
 *   token_mask  device uint8 [T], zero: masked; or NULL
 *   counts      device int32 [E]: written, or with topk_idx NULL read only, unless T
 *               is 0;  mean_prob device fp32 [E] or NULL
 *   losses      device fp32 [2] or NULL
 *   d_loss      device fp32 [1] or NULL (one): the losses' gradient, such as a
 *               loss scale
 *   dlogits     device [T] rows of E values of dlogits_dtype, ldd apart, or NULL;
 *               must not overlap logits
 *   ws          device scratch of moe_balance_loss_workspace_bytes(T, E) bytes (may
 *               be 0), 16-byte aligned, no initialisation; calls that share it must
 *               not overlap
 * Counts are exact, sums fp32 in an order that depends on T and E only.
 * Errors: MOE_EINVAL for bad sizes, types, coefficients that are not finite, null
 * or misaligned pointers; MOE_EUNSUPPORTED for E > 1024 or T*k >= 2^31; MOE_ENOMEM.
 * No choice counted, or given counts of zero: the balance loss and its gradient are
 * zero.  Every token masked: everything is zero but given counts, which stay.  T = 0:
 * everything is set to zero, counts too, also where topk_idx is NULL (counts summed up
 * over several calls are not passed to one without tokens).
 */
size_t moe_balance_loss_workspace_bytes(int T, int E);
int moe_balance_loss(const void *logits, int logits_dtype, int64_t ld, const int32_t *topk_idx,
                     const uint8_t *token_mask, int T, int E, int k, int score, float coef,
                     float z_coef, int32_t *counts, float *mean_prob, float *losses,
                     const float *d_loss, void *dlogits, int dlogits_dtype, int64_t ldd, void *ws,
                     size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------- expert slot pool */
/*
 * Partial residency (Horizon RunMap "03 / Arquitetura",
 * resident-qpacked-cache-v1; "07 / De volta à oficina": hit, miss, discard):
 * the complete INT4 source stays immutable in pinned host memory; each layer
 * owns C resident slots plus S spare slots in HBM; a miss is copied into a
 * spare slot on a side stream while readers keep the previous generation;
 * once the routed group's copies complete, a new complete generation of the
 * layer's expert table is published; an evicted slot is reused only after
 * the kernels that read it have retired.  Capacity is fixed at creation.
 * Eviction (Strata, decayed access counter; reading): per routed event of a
 * layer, every counter of the layer decays c <- c - (c >> decay_shift)
 * (decay_shift < 0: no decay), routed experts add 65536, hits then misses
 * are touched in ascending id on a use clock, and each miss (ascending id)
 * evicts the resident non-routed expert with the lowest (counter, last use,
 * id).  decay_shift = 0 is plain LRU.  Initial placement: experts 0..C-1.
 */
typedef struct moe_pool *moe_pool_t;

typedef struct {
    int layers;            /* L */
    int experts;           /* E per layer */
    int topk;              /* k */
    int capacity;          /* C resident slots per layer, k <= C <= E */
    int spares;            /* S spare slots per layer, S >= k */
    int decay_shift;       /* counter decay; < 0 disables decay */
    int64_t expert_bytes;  /* bytes of one prepacked blob */
} moe_pool_config;

typedef struct {
    int64_t hits, misses, evictions, h2d_bytes, generation;
} moe_pool_stats_t;

/*
 * pinned_src: host array of L*E host pointers (index l*E + e), each a blob
 * in device layout inside pinned host memory (hipHostMalloc); read-only.
 * Allocates L*(C+S) slots and 2*L tables of E device pointers on the
 * current device, a side stream and events, and uploads the initial
 * placement (synchronously).  MOE_ECAPACITY if C < k, C > E, S < k, or the
 * slots do not fit in free device memory; MOE_EINVAL on bad arguments.
 */
int moe_pool_create(const moe_pool_config *cfg, const void *const *pinned_src,
                    moe_pool_t *out);

/*
 * Make the distinct experts among host_ids[0..n) (the layer's routed ids,
 * copied to the host) resident and publish the layer's next generation.
 * Misses are copied H2D on the side stream into spare slots (waiting for the
 * retirement of earlier readers of those slots); the compute stream is made
 * to wait for the copies and the table update (a call whose experts are all
 * resident republishes the current table: nothing copied, nothing awaited).
 * *d_table_out receives the
 * device array of E blob pointers to pass to moe_expert_ffn_w4a16 on
 * `compute` (NULL for non-resident experts).  `step` (may be NULL) gets this
 * call's counters (hits/misses/evictions/h2d_bytes; generation = new one).
 * MOE_ECAPACITY if the routed set has more misses than spares or more
 * distinct experts than C; MOE_ESTATE if the layer's previous generation was
 * not retired.  On any error the previous generation and all counters are
 * unchanged.
 */
int moe_pool_prepare(moe_pool_t pool, int layer, const int32_t *host_ids, int n,
                     hipStream_t compute, const void *const **d_table_out,
                     moe_pool_stats_t *step);

/*
 * Profile-pinned policy for one layer (local-inference explainer,
 * lucashiago.com.br, step 4: besides keeping what was used last, one can
 * measure usage first and fix the most used experts; such a profile ages when
 * the workload changes).  experts[0..n): host int32, n must equal C, distinct
 * ids in [0, E) -- typically the C most frequent experts of a measured
 * profile.  They are copied into the layer's C resident slots (synchronously;
 * the call waits for the device) and stay there: from now on a routed expert
 * of the set is a hit, and every other routed expert is a miss copied into a
 * spare slot for that generation only, dropped at the layer's next prepare
 * (paid again at its next use; nothing is evicted, evictions stay 0).
 * moe_pool_reset() returns every layer to the decayed-counter policy and the
 * canonical placement.  MOE_EINVAL on bad ids or n != C; MOE_ESTATE if the
 * layer's last generation was not retired.
 */
int moe_pool_pin(moe_pool_t pool, int layer, const int32_t *experts, int n);

/* Record that every kernel enqueued on `compute` so far that reads the
 * layer's current generation has been issued; slots evicted by it become
 * reusable once those kernels finish.  MOE_ESTATE if nothing to retire. */
int moe_pool_retire(moe_pool_t pool, int layer, hipStream_t compute);

/*
 * One pooled MoE layer for a small batch -- the decode loop of a partially
 * resident model -- in one host call, with the same readings as the calls it
 * chains: moe_route_permute on `stream`; the T*k routed ids copied into
 * host_ids (pinned host memory) and waited for (this call blocks the calling
 * thread until they arrive; for one token of at most 64 experts the routing
 * kernel itself writes them, then a sequence flag, into the pool's own
 * coherent pinned buffer and the thread spins on the flag, MOE_EHIP after
 * 10 s, instead of a device-to-host copy and an event wait); moe_pool_prepare
 * on this layer; the routed
 * expert FFN (moe_expert_ffn_w4a16 with the published table and `regime`);
 * moe_pool_retire; moe_combine into out_f16.  E is the pool's expert count.
 * When the routed set has both hits and misses and the decode kernel runs,
 * the hits are computed first, on the previous generation's table (where
 * every hit already sits in its slot and no miss appears), while the misses
 * are copied; a second launch on the new table then computes the misses.
 * Every buffer is the caller's, sized as for those calls (route_ws:
 * moe_route_permute_workspace_bytes, zero-filled before its first use;
 * y / ffn_ws: moe_expert_ffn_plan).  Errors are those of the chained calls;
 * the first one stops the chain (a failure in prepare leaves the layer's
 * previous generation published).
 */
typedef struct {
    const void *x_f16;          /* device fp16 [T][H] */
    const void *w_router_f16;   /* device fp16 [E][H] */
    const float *logit_bias;    /* device fp32 [E] or NULL */
    int T, H, I, k, group;
    unsigned flags;             /* MOE_RENORM or 0 */
    int32_t *topk_idx;          /* device [T][k] */
    float *topk_w;              /* device [T][k] */
    int32_t *counts, *offsets, *perm, *inv_perm;   /* device, as moe_permute */
    void *route_ws;
    size_t route_ws_bytes;
    int regime;                 /* MOE_REGIME_* */
    void *y;
    int y_dtype, y_slices;
    void *ffn_ws;
    size_t ffn_ws_bytes;
    const float *shared_f32;    /* device fp32 [T][H] or NULL */
    const void *residual_f16;   /* device fp16 [T][H] or NULL */
    void *out_f16;              /* device fp16 [T][H] */
    int32_t *host_ids;          /* pinned host int32 [T*k] */
} moe_pool_layer_args;

int moe_pool_layer_forward(moe_pool_t pool, int layer, const moe_pool_layer_args *args,
                           hipStream_t stream, moe_pool_stats_t *step);

/* Cumulative counters since creation or the last reset. */
int moe_pool_stats(moe_pool_t pool, moe_pool_stats_t *out);

/*
 * Per-(layer, expert) access counts since creation or the last reset: the
 * uses of each expert that found it resident and those that copied it in.
 * Their sum over a layer is that layer's routed distinct experts over all
 * its generations.  This is the data a live map of expert traffic is drawn
 * from (Strata, "Tracking MoE expert residency": aggregate hit rates did not
 * explain the behaviour; the per-layer, per-expert distribution did).
 * hits, misses: host int64 arrays of layers*experts, index l*E + e, written.
 * MOE_EINVAL on a null argument.  Host only: nothing waits for the device.
 */
int moe_pool_access_counts(moe_pool_t pool, int64_t *hits, int64_t *misses);

/* Waits for all pool work, restores the initial placement, clears counters. */
int moe_pool_reset(moe_pool_t pool);

/* Waits for all pool work and frees everything.  NULL is a no-op. */
int moe_pool_destroy(moe_pool_t pool);

#ifdef __cplusplus
}
#endif

#endif /* MOE_W4A16_H */
