"""Plumbing around the C ABI: device buffers (torch) and the call sequence of
one MoE layer -- route, permute, routed expert FFN, optional shared expert,
combine.  No arithmetic happens here; every step is a libmoe_w4a16 call on
the given stream.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _abi as A


def load_experts(weights, H, I, group, device="cuda", stream=None, fmt=A.MOE_FMT_SYM):
    """Quantise and prepack experts on the device.

    weights: iterable of (wg [I,H], wu [I,H], wd [H,I]) float32 arrays
    (numpy or torch).  Returns a uint8 device tensor [n, blob_bytes] in the
    device layout (and the canonical blobs).  Quantisation and prepacking run
    in the library's kernels; fmt is MOE_FMT_SYM or MOE_FMT_ZP.
    """
    weights = list(weights)
    n = len(weights)
    _, total = A.moe_blob_layout_fmt(H, I, group, fmt)
    dev = torch.empty((n, total), dtype=torch.uint8, device=device)
    canon = torch.empty((n, total), dtype=torch.uint8, device=device)
    wg = torch.empty((n, I, H), dtype=torch.float32, device=device)
    wu = torch.empty((n, I, H), dtype=torch.float32, device=device)
    wd = torch.empty((n, H, I), dtype=torch.float32, device=device)
    for e, (g_, u_, d_) in enumerate(weights):
        wg[e].copy_(torch.as_tensor(g_))
        wu[e].copy_(torch.as_tensor(u_))
        wd[e].copy_(torch.as_tensor(d_))
    A.moe_quantize_experts_fmt(wg, wu, wd, n, H, I, group, fmt, canon, stream)
    A.moe_prepack_experts_fmt(canon, n, H, I, group, fmt, dev, stream)
    return dev, canon


def load_experts_fp8(weights, H, I, device="cuda", stream=None):
    """Quantise experts to e4m3 with a scale per 128 x 128 block on the device.

    weights: iterable of (wg [I,H], wu [I,H], wd [H,I]) float32 arrays (numpy
    or torch).  Returns a uint8 device tensor [n, blob_bytes] in the layout of
    moe_fp8_blob_layout, which the kernels read as it is.  ValueError for an
    expert that is not three matrices of these shapes.  The copies are made on
    the device's current stream; with a stream of its own (an object or an
    address) the quantisation waits for them there, and the current stream for
    it, without the host."""
    shapes = ((I, H), (I, H), (H, I))
    weights = [tuple(w) for w in weights]
    for e, w in enumerate(weights):   # the quantiser sees addresses, not shapes
        got = tuple(tuple(torch.as_tensor(m).shape) for m in w)
        if got != shapes:
            raise ValueError("expert %d: matrices of shapes %s, expected %s" % (e, got, shapes))
    off, total = A.moe_fp8_blob_layout(H, I)
    blobs = torch.zeros((len(weights), total), dtype=torch.uint8, device=device)
    with torch.cuda.device(blobs.device):   # the library launches on the current device
        here = torch.cuda.current_stream()
        there = here if stream is None else _stream_object(stream)
        for e, w in enumerate(weights):
            base = blobs[e].data_ptr()
            for j, (m, (rows, cols)) in enumerate(zip(w, shapes)):
                m = torch.as_tensor(m).to(device=blobs.device, dtype=torch.float32).contiguous()
                there.wait_stream(here)
                A.moe_quantize_fp8(m, A.MOE_DTYPE_F32, cols, rows, cols, 128, 0, base + off[j],
                                   cols, base + off[3 + j], there)
                here.wait_stream(there)   # m's memory goes to later work of this stream
    return blobs


def _stream_object(stream):
    """A torch stream of the current device for a stream given as such or as
    an address (0: the default stream)."""
    if not isinstance(stream, int):
        return stream
    return torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()


@dataclass
class ScoreRouting:
    """Expert selection by moe_route_select instead of moe_route's softmax
    top-k: scores (MOE_SCORE_*), a bias that decides but does not weigh, expert
    groups of which topk_group are kept, and a factor on the weights."""
    score: int = A.MOE_SCORE_SIGMOID
    select_bias: torch.Tensor | None = None   # fp32 [E] device
    n_group: int = 1
    topk_group: int = 1
    group_top2: bool = False                  # a group counts by its two best experts
    scale: float = 1.0


def _types(*weights):
    return {w.dtype for w in weights if w is not None}


def _w_dtype(types):
    return A.MOE_DTYPE_F32 if torch.float32 in types else A.MOE_DTYPE_F16


@dataclass
class BlockNorms:
    """The norms, gate and residual scale around a layer's block (moe_block_norm):
    h' = h + scale * gate * post(MoE(pre(h))).  Weights fp16 or fp32 [H] device (all
    of one type, in a stack too; any may be absent), gate fp16 [H] device."""
    pre_w: torch.Tensor | None = None
    pre_b: torch.Tensor | None = None
    post: bool = False                        # norm the block's output too
    post_w: torch.Tensor | None = None
    post_b: torch.Tensor | None = None
    gate: torch.Tensor | None = None
    scale: float = 1.0
    kind: int = A.MOE_NORM_RMS
    eps: float = 1e-5
    unit_offset: bool = False                 # weights count as 1 + w

    def __post_init__(self):
        if len(self.types) > 1 or self.types - {torch.float16, torch.float32}:
            raise ValueError("norm weights must all be fp16 or all fp32")

    @property
    def types(self):
        """Types of the weights that there are."""
        return _types(self.pre_w, self.pre_b, self.post_w, self.post_b)

    @property
    def w_dtype(self):
        return _w_dtype(self.types)

    def check(self, H):
        """ValueError where a weight or the gate is not of rows of H."""
        for w in (self.pre_w, self.pre_b, self.post_w, self.post_b, self.gate):
            if w is not None and (w.numel() != H or not w.is_contiguous()):
                raise ValueError("norm weights and gates must be contiguous, of %d values" % H)
        if self.gate is not None and self.gate.dtype != torch.float16:
            raise ValueError("the gate must be fp16")
        if not self.post and (self.post_w is not None or self.post_b is not None):
            raise ValueError("post-norm weights without post")

    @property
    def form(self):
        """What the norms of a stack have in common."""
        return self.kind, self.eps, self.unit_offset


def block_norm(y, h, end, start, out, n, stream=None):
    """The end of one block and the start of the next on fp16 rows: out = h +
    scale * gate * post(y) as `end` says (None: there is no block, y is None) and n =
    pre(out) as `start` says (None: n is None).  One moe_block_norm call."""
    norms = end if start is None else start
    if end is not None and start is not None:
        if end.form != start.form:
            raise ValueError("the norms of a stack must have one kind, eps and unit_offset")
    T, H = h.shape
    flags = A.MOE_NORM_UNIT_OFFSET if norms.unit_offset else 0
    gate = post_w = post_b = None
    scale = 1.0
    if end is not None:
        gate, scale = end.gate, end.scale
        if end.post:
            post_w, post_b, flags = end.post_w, end.post_b, flags | A.MOE_NORM_POST
    pre_w, pre_b = (None, None) if start is None else (start.pre_w, start.pre_b)
    types = _types(post_w, post_b, pre_w, pre_b)
    if len(types) > 1:
        raise ValueError("the norms of a stack must have weights of one type")
    A.moe_block_norm(y, H, h, H, gate, 0, scale, post_w, post_b, pre_w, pre_b, A.MOE_DTYPE_F16,
                     _w_dtype(types), norms.kind, flags, norms.eps, T, H, out, H, n, H, stream)


def blob_table(blobs: torch.Tensor) -> torch.Tensor:
    """Device array of per-expert blob addresses for a [E, bytes] tensor."""
    E, nbytes = blobs.shape
    base = blobs.data_ptr()
    return torch.tensor([base + e * nbytes for e in range(E)], dtype=torch.int64,
                        device=blobs.device)


@dataclass
class LayerBuffers:
    T: int
    regime: int
    y_dtype: int
    y_slices: int
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    perm: torch.Tensor
    inv_perm: torch.Tensor
    perm_ws: torch.Tensor | None
    y: torch.Tensor
    ffn_ws: torch.Tensor | None
    shared_out: torch.Tensor | None
    shared_ws: torch.Tensor | None
    out: torch.Tensor
    logits: torch.Tensor | None = None
    router_ws: torch.Tensor | None = None
    normed: torch.Tensor | None = None


@dataclass
class BalanceBuffers:
    """What MoELayer.balance and router_backward write (MoELayer.balance_buffers)."""
    logits: torch.Tensor       # fp32 [T, E]: the router's, where the routing keeps none
    counts: torch.Tensor       # int32 [E]
    mean_prob: torch.Tensor    # fp32 [E]
    losses: torch.Tensor       # fp32 [2]: balance loss, z loss
    dlogits: torch.Tensor      # fp16 [T, E], times balance's d_loss
    d_router: torch.Tensor     # fp32 [E, H]
    d_bias: torch.Tensor       # fp32 [E]
    dx: torch.Tensor           # fp32 [T, H]
    ws: torch.Tensor
    formed: bool = False       # whether the last balance call formed dlogits


class MoELayer:
    """One MoE layer resident on the device: W4A16 experts (fmt MOE_FMT_SYM or
    MOE_FMT_ZP) or FP8 experts (MOE_FMT_FP8: blobs of load_experts_fp8, `group`
    unused), routed by softmax top-k or, with `routing`, by scores and groups.
    The softmax router takes H in {256, 512, 1024, 2048}; with `routing` the
    logits of other H come from moe_linear_f16 (any multiple of 8).  `norms`: the
    norms around the block, which stack_forward applies, also to a stack of one
    layer; forward and the other methods of a layer are the block itself."""

    def __init__(self, H, I, E, k, group, router, table, bias=None, shared=None,
                 renorm=False, device="cuda", shared_gate=None, overlap_shared=False,
                 fmt=A.MOE_FMT_SYM, routing: ScoreRouting | None = None,
                 norms: BlockNorms | None = None):
        self.H, self.I, self.E, self.k, self.g = H, I, E, k, group
        self.fmt = fmt                  # blob format of the routed experts
        self.router = router            # fp16 [E, H] device
        self.table = table              # int64 [E] device (blob addresses)
        self.bias = bias                # fp32 [E] device or None
        self.shared = shared            # (wg, wu, wd) fp16 device or None
        self.shared_gate = shared_gate  # fp16 [H] device or None (sigmoid-gated shared)
        # run the shared expert on a side stream next to routing + routed FFN
        self.overlap_shared = overlap_shared
        if shared_gate is not None and shared is None:
            raise ValueError("a shared-expert gate needs a shared expert")
        self.flags = A.MOE_RENORM if renorm else 0
        self.routing = routing
        if norms is not None:
            norms.check(H)
        self.norms = norms
        self.device = device

    @property
    def fp8(self) -> bool:
        return self.fmt == A.MOE_FMT_FP8

    def buffers(self, T, regime=A.MOE_REGIME_AUTO, partial_order=True) -> LayerBuffers:
        """partial_order: decode partials in partial-major column order, which
        the fused combine + next route reads in whole lines.  FP8 layers:
        regime may carry MOE_ACC_F32 (fp32 sums in every product)."""
        d = self.device
        if self.fp8:
            r, ffn_ws = A.moe_expert_ffn_w8a8_plan(T, self.H, self.I, self.E, self.k, regime)
            ydt, ysl = A.MOE_DTYPE_F16, 1
        else:
            r, ydt, ysl, ffn_ws = A.moe_expert_ffn_plan(T, self.H, self.I, self.E, self.k, self.g,
                                                        regime)
        if not self.fp8 and r == A.MOE_REGIME_DECODE:
            # decode partials straight in token order: the combine then reads
            # them without inv_perm (one dependent round trip less)
            r |= A.MOE_Y_TOKEN_ORDER
            if partial_order and (self.H // 8 <= 64 or (self.H // 8) % 64 == 0):
                r |= A.MOE_Y_PARTIAL_ORDER
                ydt = A.moe_expert_ffn_plan(T, self.H, self.I, self.E, self.k, self.g, r)[1]
        if self.fmt == A.MOE_FMT_ZP:
            r |= A.MOE_W4_ZERO_POINT
        # route/permute scratch; zero-filled once (the fused router keeps an
        # atomic ticket in it)
        pws = max(A.moe_permute_workspace_bytes(T, self.k, self.E),
                  A.moe_route_permute_workspace_bytes(T, self.k, self.E),
                  A.moe_combine_route_permute_workspace_bytes(T, self.k, self.E))
        logits = router_ws = normed = None
        if self.routing is not None:
            pws = max(pws, A.moe_route_select_workspace_bytes(T, self.k, self.E))
            logits = torch.empty((T, self.E), dtype=torch.float32, device=d)
            if not self.pinned_router:
                n = A.moe_linear_f16_workspace_bytes(T, self.E, self.H)
                router_ws = torch.empty(n, dtype=torch.uint8, device=d) if n else None
        if self.norms is not None:
            normed = torch.empty((T, self.H), dtype=torch.float16, device=d)
        n = T * self.k
        ytype = torch.float16 if ydt == A.MOE_DTYPE_F16 else torch.float32
        sh_out = sh_ws = None
        if self.shared is not None:
            Is = self.shared[0].shape[0]
            sh_out = torch.empty((T, self.H), dtype=torch.float32, device=d)
            # zero-filled once: the split-K reduction keeps arrival counters
            # in it and leaves them zero after every call
            sh_ws = torch.zeros(max(1, A.moe_shared_ffn_workspace_bytes(T, self.H, Is)),
                                dtype=torch.uint8, device=d)
        return LayerBuffers(
            T=T, regime=r, y_dtype=ydt, y_slices=ysl,
            topk_idx=torch.empty((T, self.k), dtype=torch.int32, device=d),
            topk_w=torch.empty((T, self.k), dtype=torch.float32, device=d),
            counts=torch.empty(self.E, dtype=torch.int32, device=d),
            offsets=torch.empty(self.E + 1, dtype=torch.int32, device=d),
            perm=torch.empty(max(n, 1), dtype=torch.int32, device=d),
            inv_perm=torch.empty(max(n, 1), dtype=torch.int32, device=d),
            perm_ws=torch.zeros(pws, dtype=torch.uint8, device=d) if pws else None,
            y=torch.empty((ysl, max(n, 1), self.H), dtype=ytype, device=d),
            ffn_ws=torch.empty(ffn_ws, dtype=torch.uint8, device=d) if ffn_ws else None,
            shared_out=sh_out, shared_ws=sh_ws,
            out=torch.empty((T, self.H), dtype=torch.float16, device=d),
            logits=logits, router_ws=router_ws, normed=normed,
        )

    @property
    def pinned_router(self) -> bool:
        """Whether the router's logits have the pinned summation order (moe_route's)."""
        return self.H in (256, 512, 1024, 2048)

    def router_logits(self, x, logits, ws=None, stream=None):
        """The router's fp32 logits [T, E] of x."""
        T = logits.shape[0]
        if self.pinned_router:
            A.moe_router_logits(x, self.router, self.bias, T, self.H, self.E, logits, stream)
            return
        A.moe_linear_f16(x, self.H, self.router, self.H, self.bias, A.MOE_ACT_NONE, None, 0, T,
                         self.E, self.H, logits, A.MOE_DTYPE_F32, self.E, None, 0, ws,
                         0 if ws is None else ws.numel(), stream)

    def route_permute(self, x, b: LayerBuffers, stream=None, fused=True):
        T = b.T
        nws = 0 if b.perm_ws is None else b.perm_ws.numel()
        if self.routing is not None:
            s = self.routing
            self.router_logits(x, b.logits, b.router_ws, stream)
            A.moe_route_select_permute(
                b.logits, A.MOE_DTYPE_F32, self.E, s.select_bias, T, self.E, self.k, s.score,
                s.n_group, s.topk_group, self.flags | (A.MOE_GROUP_TOP2 if s.group_top2 else 0),
                s.scale, b.topk_idx, b.topk_w, b.counts, b.offsets, b.perm, b.inv_perm, b.perm_ws,
                nws, stream)
            return
        if fused:
            A.moe_route_permute(x, self.router, self.bias, T, self.H, self.E, self.k,
                                self.flags, b.topk_idx, b.topk_w, b.counts, b.offsets, b.perm,
                                b.inv_perm, b.perm_ws, nws, stream)
            return
        A.moe_route(x, self.router, self.bias, T, self.H, self.E, self.k, self.flags,
                    b.topk_idx, b.topk_w, b.perm_ws, nws, stream)
        A.moe_permute(b.topk_idx, T, self.k, self.E, b.counts, b.offsets, b.perm, b.inv_perm,
                      b.perm_ws, nws, stream)

    def shared_ffn(self, x, b: LayerBuffers, stream=None):
        wg, wu, wd = self.shared
        A.moe_shared_ffn_f16(x, wg, wu, wd, b.T, self.H, wg.shape[0], b.shared_out,
                             b.shared_ws, b.shared_ws.numel(), stream)

    def experts(self, x, b: LayerBuffers, table=None, stream=None, shared=True):
        if self.fp8:
            A.moe_expert_ffn_w8a8(x, b.perm, b.offsets, self.table if table is None else table,
                                  b.T, self.H, self.I, self.E, self.k, b.regime, b.y, b.ffn_ws,
                                  0 if b.ffn_ws is None else b.ffn_ws.numel(), stream)
            if shared and self.shared is not None:
                self.shared_ffn(x, b, stream)
            return
        A.moe_expert_ffn_w4a16(x, b.perm, b.offsets, self.table if table is None else table,
                               b.T, self.H, self.I, self.E, self.k, self.g, b.regime, b.y,
                               b.y_dtype, b.y_slices, b.ffn_ws,
                               0 if b.ffn_ws is None else b.ffn_ws.numel(), stream)
        if shared and self.shared is not None:
            self.shared_ffn(x, b, stream)

    def combine(self, b: LayerBuffers, residual=None, out=None, stream=None, x=None):
        """x (the layer input) is needed only when the shared expert is gated."""
        out = b.out if out is None else out
        inv = None if b.regime & A.MOE_Y_TOKEN_ORDER else b.inv_perm
        if self.shared_gate is not None:
            if x is None:
                raise ValueError("the gated shared expert needs the layer input x")
            A.moe_combine_gated(b.y, b.y_dtype, b.y_slices, inv, b.topk_w, b.shared_out,
                                x, self.shared_gate, residual, b.T, self.H, self.k, out, stream)
            return out
        A.moe_combine(b.y, b.y_dtype, b.y_slices, inv, b.topk_w, b.shared_out, residual,
                      b.T, self.H, self.k, out, stream)
        return out

    def combine_route_next(self, b: LayerBuffers, nxt: "MoELayer", b_next: LayerBuffers,
                           residual=None, out=None, stream=None, x=None):
        """This layer's combine into `out` fused with the next layer's route +
        permute of `out` into b_next (moe_combine_route_permute: one launch for a
        decode token of at most 64 experts, else the two calls)."""
        if nxt.H != self.H or b_next.T != b.T:
            raise ValueError("the next layer must have the same H and batch")
        if nxt.routing is not None:
            raise ValueError("the fused call routes by softmax top-k only")
        out = b.out if out is None else out
        inv = None if b.regime & A.MOE_Y_TOKEN_ORDER else b.inv_perm
        gate = self.shared_gate
        if gate is not None and x is None:
            raise ValueError("the gated shared expert needs the layer input x")
        nws = 0 if b_next.perm_ws is None else b_next.perm_ws.numel()
        A.moe_combine_route_permute(b.y, b.y_dtype, b.y_slices, inv, b.topk_w, b.shared_out,
                                    x if gate is not None else None, gate, residual, b.T,
                                    self.H, self.k, out, nxt.router, nxt.bias, nxt.E, nxt.k,
                                    nxt.flags, b_next.topk_idx, b_next.topk_w, b_next.counts,
                                    b_next.offsets, b_next.perm, b_next.inv_perm, b_next.perm_ws,
                                    nws, stream)
        return out

    def split_route_ok(self, b: LayerBuffers, nxt: "MoELayer") -> bool:
        """Whether this layer's combine can hand the next layer only its logit
        partials (moe_combine_route_partials): one decode token, at most 64
        experts in the next layer, fp32 slice partials here."""
        return (b.T == 1 and nxt.E <= 64 and nxt.H == self.H and b.y_slices > 1 and
                b.y_dtype in (A.MOE_DTYPE_F32, A.MOE_DTYPE_F32_PM) and not nxt.fp8 and
                nxt.routing is None)

    def combine_partials_next(self, b: LayerBuffers, nxt: "MoELayer", parts,
                              residual=None, out=None, stream=None, x=None):
        """This layer's combine into `out` plus the next layer's logit partials
        of `out` into `parts` (fp32, moe_logit_partials_bytes()), which
        nxt.experts_routed then routes from."""
        nxt._check_partials()
        out = b.out if out is None else out
        inv = None if b.regime & A.MOE_Y_TOKEN_ORDER else b.inv_perm
        gate = self.shared_gate
        if gate is not None and x is None:
            raise ValueError("the gated shared expert needs the layer input x")
        A.moe_combine_route_partials(b.y, b.y_dtype, b.y_slices, inv, b.topk_w, b.shared_out,
                                     x if gate is not None else None, gate, residual, b.T,
                                     self.H, self.k, out, nxt.router, nxt.E, parts, stream)
        return out

    def route_from_partials_ok(self, b: LayerBuffers) -> bool:
        """Whether this layer's expert launch can route from logit partials
        (moe_expert_ffn_w4a16_routed): one decode token, at most 64 experts."""
        return (b.T == 1 and self.E <= 64 and b.regime & 0xFF == A.MOE_REGIME_DECODE and
                not self.fp8 and self.routing is None)

    def _check_partials(self):
        if self.fp8 or self.routing is not None:
            raise ValueError("routing from logit partials is for W4A16 experts and softmax top-k")

    def logit_partials(self, x, parts, stream=None):
        """This layer's logit partials of an input row in hand (the first
        layer of a stack) into `parts`, for experts_routed."""
        self._check_partials()
        A.moe_logit_partials(x, self.router, 1, self.H, self.E, parts, stream)

    def experts_routed(self, x, b: LayerBuffers, parts, stream=None, shared=True):
        """Routing from the logit partials of the previous layer's combine and
        the routed experts in one launch (moe_expert_ffn_w4a16_routed): fills
        b's routing arrays and y as route_permute + experts would.  ValueError
        for a layer with FP8 experts or score routing."""
        self._check_partials()
        A.moe_expert_ffn_w4a16_routed(x, parts, self.bias, self.E, self.k, self.flags,
                                      b.topk_idx, b.topk_w, b.counts, b.offsets, b.perm,
                                      b.inv_perm, self.table, b.T, self.H, self.I, self.g,
                                      b.regime, b.y, b.y_dtype, b.y_slices, stream)
        if shared and self.shared is not None:
            self.shared_ffn(x, b, stream)

    def balance_buffers(self, T) -> BalanceBuffers:
        d = self.device
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device=d)  # noqa: E731
        n = max(A.moe_balance_loss_workspace_bytes(T, self.E),
                A.moe_linear_f16_workspace_bytes(T, self.E, self.H),
                A.moe_linear_f16_backward_workspace_bytes(T, self.E, self.H), 1)
        return BalanceBuffers(
            logits=e(T, self.E), counts=e(self.E, t=torch.int32), mean_prob=e(self.E), losses=e(2),
            dlogits=e(T, self.E, t=torch.float16), d_router=e(self.E, self.H), d_bias=e(self.E),
            dx=e(T, self.H), ws=e(n, t=torch.uint8))

    def _check_balance(self, x, g: BalanceBuffers):
        """ValueError for buffers of other layers, and for x of other rows than theirs."""
        if g.d_router.shape != (self.E, self.H):
            raise ValueError("balance buffers of %d experts of %d, not %d of %d" %
                             (*g.d_router.shape, self.E, self.H))
        if x.numel() != g.dx.numel() or x.shape[-1] != self.H:
            raise ValueError("x must hold %d rows of %d" % g.dx.shape)

    def balance(self, x, b: LayerBuffers, g: BalanceBuffers, coef, z_coef=0.0, mask=None,
                d_loss=None, stream=None):
        """After route_permute of x into b: the routing's balance loss, z loss, counts
        and mean probabilities over the tokens that `mask` (uint8 [T], zero: padding)
        leaves, and with d_loss (fp32 [1] device) the logits' gradient times it, into g.
        That gradient is fp16, and by itself mostly below fp16's smallest step (coef 0.01
        over 4096 tokens and 64 experts: 5e-8 at most): d_loss is a loss scale, such as
        65536, which router_backward's results carry.  Without it no gradient is formed.
        Scores as the layer's router forms them, without the selection's bias.  Returns
        g.losses."""
        if g.dlogits.shape[0] != b.T:
            raise ValueError("balance buffers of %d tokens, not %d" % (g.dlogits.shape[0], b.T))
        self._check_balance(x, g)
        if mask is not None and (mask.numel() != b.T or mask.element_size() != 1
                                 or not mask.is_contiguous()):
            raise ValueError("the mask must hold %d bytes" % b.T)
        if d_loss is not None and (d_loss.dtype != torch.float32 or d_loss.numel() != 1):
            raise ValueError("d_loss must be one fp32 value")
        if any(t is not None and t.device != x.device for t in (mask, d_loss)):
            raise ValueError("the mask and d_loss must be on the device of x")
        logits = b.logits
        if logits is None:
            logits = g.logits
            self.router_logits(x, logits, g.ws, stream)
        score = A.MOE_SCORE_SOFTMAX if self.routing is None else self.routing.score
        A.moe_balance_loss(logits, A.MOE_DTYPE_F32, self.E, b.topk_idx, mask, b.T, self.E, self.k,
                           score, coef, z_coef, g.counts, g.mean_prob, g.losses, d_loss,
                           None if d_loss is None else g.dlogits, A.MOE_DTYPE_F16, self.E, g.ws,
                           g.ws.numel(), stream)
        g.formed = d_loss is not None
        return g.losses

    def router_backward(self, x, g: BalanceBuffers, stream=None):
        """Gradients of the router's weights, of its bias and of x from g.dlogits (from
        balance), into g.d_router, g.d_bias and g.dx: fp32, times balance's d_loss.
        ValueError where the last balance call had none."""
        self._check_balance(x, g)
        if not g.formed:
            raise ValueError("no gradient to go back from: balance was given no d_loss")
        A.moe_linear_f16_backward(g.dlogits, self.E, None, 0, A.MOE_ACT_NONE, x, self.H,
                                  self.router, self.H, g.dlogits.shape[0], self.E, self.H, g.dx,
                                  self.H, g.d_router, self.H, A.MOE_DTYPE_F32, g.d_bias, g.ws,
                                  g.ws.numel(), stream)

    def pool_args(self, b: LayerBuffers, host_ids):
        """PoolLayerArgs for moe_pool_layer_forward with this layer's weights and
        b's buffers; x_f16 / residual_f16 / out_f16 are set per call."""
        if self.shared is not None:
            raise ValueError("pooled layers carry no shared expert")
        if self.fp8 or self.routing is not None or self.norms is not None:
            raise ValueError("pooled layers are W4A16 with the softmax router, without norms")
        z = lambda t: 0 if t is None else t.data_ptr()
        a = A.PoolLayerArgs()
        a.w_router_f16, a.logit_bias = z(self.router), z(self.bias)
        a.T, a.H, a.I, a.k, a.group, a.flags = b.T, self.H, self.I, self.k, self.g, self.flags
        a.topk_idx, a.topk_w, a.counts = z(b.topk_idx), z(b.topk_w), z(b.counts)
        a.offsets, a.perm, a.inv_perm = z(b.offsets), z(b.perm), z(b.inv_perm)
        a.route_ws, a.route_ws_bytes = z(b.perm_ws), 0 if b.perm_ws is None else b.perm_ws.numel()
        a.regime, a.y, a.y_dtype, a.y_slices = b.regime, z(b.y), b.y_dtype, b.y_slices
        a.ffn_ws, a.ffn_ws_bytes = z(b.ffn_ws), 0 if b.ffn_ws is None else b.ffn_ws.numel()
        a.host_ids = host_ids.data_ptr()
        return a

    def _side(self):
        st = getattr(self, "_side_stream", None)
        if st is None:
            st = self._side_stream = torch.cuda.Stream(device=self.device)
        return st

    def forward(self, x, b: LayerBuffers, residual=None, out=None, stream=None,
                overlap_shared=None):
        """One layer's block, of x as it is (its `norms` are stack_forward's).
        With overlap_shared (default: the layer's setting) the shared expert
        runs on a side stream, forked at the layer's start and joined before
        the combine: it reads only x, so it overlaps routing and the routed
        experts.  That pays when the shared weights are large
        (60-expert layer, 69 MB: -12% per layer at T = 8..256) and costs when
        they are small (512-expert layer, 6 MB: +17% at T = 1, the shared
        kernels then delay the latency-bound router)."""
        if overlap_shared is None:
            overlap_shared = self.overlap_shared
        if self.shared is None or not overlap_shared or isinstance(stream, int):
            self.route_permute(x, b, stream)
            self.experts(x, b, stream=stream)
            return self.combine(b, residual, out, stream, x=x)
        main = torch.cuda.current_stream(self.device) if stream is None else stream
        side = self._side()
        fork = torch.cuda.Event()
        fork.record(main)
        side.wait_event(fork)
        if not torch.cuda.is_current_stream_capturing():
            x.record_stream(side)
        self.shared_ffn(x, b, side)
        join = torch.cuda.Event()
        join.record(side)
        self.route_permute(x, b, main)
        self.experts(x, b, stream=main, shared=False)
        main.wait_event(join)
        return self.combine(b, residual, out, main, x=x)


def stack_forward(layers, bufs, acts, stream=None, fuse=True, parts=None):
    """Stacked layers with residual connections, x_{l+1} = fp16(x_l + MoE_l(x_l)):
    acts[l] is layer l's input and residual, acts[l + 1] its output.  With
    `fuse`, each layer's combine runs together with the next layer's route +
    permute (MoELayer.combine_route_next); with `parts` as well (fp32 device
    buffer of moe_logit_partials_bytes()), a decode token's combine hands the
    next layer only its logit partials and that layer's expert launch routes
    from them (combine_partials_next + experts_routed), the first layer's
    from moe_logit_partials of its input.  Every form gives the same bits.

    Layers with `norms` (all of the stack or none; ValueError otherwise) compute
    x_{l+1} = x_l + scale_l * gate_l * post_l(MoE_l(pre_l(x_l))): the end of a block
    and the start of the next are one moe_block_norm call between a layer's combine
    and the next layer's routing, which then are not fused (`fuse` and `parts` do not
    apply); MoE_l's output is rounded to fp16 between the two calls."""
    L = len(layers)
    if any(lay.norms is not None for lay in layers):
        return _stack_normed(layers, bufs, acts, stream)
    # routed: this layer's routing is still to be formed from `parts`
    routed = fuse and parts is not None and layers[0].route_from_partials_ok(bufs[0])
    if routed:
        layers[0].logit_partials(acts[0], parts, stream)
    else:
        layers[0].route_permute(acts[0], bufs[0], stream)
    for l, lay in enumerate(layers):
        # a layer routed by scores is routed on its own, never with a combine
        if l > 0 and (not fuse or lay.routing is not None):
            lay.route_permute(acts[l], bufs[l], stream)
        if routed:
            lay.experts_routed(acts[l], bufs[l], parts, stream=stream)
        else:
            lay.experts(acts[l], bufs[l], stream=stream)
        routed = False
        if fuse and l + 1 < L and layers[l + 1].routing is None:
            nxt = layers[l + 1]
            if parts is not None and lay.split_route_ok(bufs[l], nxt) and \
                    bufs[l + 1].regime & 0xFF == A.MOE_REGIME_DECODE:
                lay.combine_partials_next(bufs[l], nxt, parts, residual=acts[l],
                                          out=acts[l + 1], stream=stream, x=acts[l])
                routed = True
            else:
                lay.combine_route_next(bufs[l], nxt, bufs[l + 1], residual=acts[l],
                                       out=acts[l + 1], stream=stream, x=acts[l])
        else:
            lay.combine(bufs[l], residual=acts[l], out=acts[l + 1], stream=stream, x=acts[l])
    return acts[L]


def _stack_normed(layers, bufs, acts, stream):
    if any(lay.norms is None for lay in layers):
        raise ValueError("a stack's layers must all have norms, or none")
    # before anything is launched
    if len({lay.norms.form for lay in layers}) > 1 or \
            len(set().union(*(lay.norms.types for lay in layers))) > 1:
        raise ValueError("the norms of a stack must have one kind, eps, unit_offset and "
                         "weights of one type")
    L = len(layers)
    block_norm(None, acts[0], None, layers[0].norms, None, bufs[0].normed, stream)
    for l, lay in enumerate(layers):
        b = bufs[l]
        lay.route_permute(b.normed, b, stream)
        lay.experts(b.normed, b, stream=stream)
        lay.combine(b, stream=stream, x=b.normed)
        last = l + 1 == L
        block_norm(b.out, acts[l], lay.norms, None if last else layers[l + 1].norms, acts[l + 1],
                   None if last else bufs[l + 1].normed, stream)
    return acts[L]
