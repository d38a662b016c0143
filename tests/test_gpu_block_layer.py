"""Layers with norms around them, routers of other widths, and a router's training
step: the operators together, as MoELayer calls them."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
from int4_weight_only_router_amd.layer import (BlockNorms, MoELayer, ScoreRouting, blob_table,
                                               load_experts, load_experts_fp8, stack_forward)
from tests import block_util as B
from tests import fp8_util as R
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
STEPS = 64   # as in test_gpu_block_norm


def half(r, *s, scale=1.0):
    return torch.from_numpy((scale * r.normal(0, 1, s)).astype(np.float16)).to(DEV)


def layer(r, H, I, E, k, routing, norms, fp8):
    w = [tuple(r.normal(0, 0.02, s).astype(np.float32) for s in ((I, H), (I, H), (H, I)))
         for _ in range(E)]
    blobs = load_experts_fp8(w, H, I, DEV) if fp8 else load_experts(w, H, I, 64, DEV)[0]
    lay = MoELayer(H, I, E, k, 0 if fp8 else 64, half(r, E, H, scale=0.05), blob_table(blobs),
                   torch.from_numpy(r.normal(0, 0.1, E).astype(np.float32)).to(DEV), device=DEV,
                   fmt=M.MOE_FMT_FP8 if fp8 else M.MOE_FMT_SYM, routing=routing, norms=norms)
    lay._blobs = blobs
    return lay


def norms(r, H, kind, post, gate, offset=False):
    base = 0.0 if offset else 1.0
    w = lambda: base + half(r, H, scale=0.1)  # noqa: E731
    return BlockNorms(w(), half(r, H, scale=0.1), post, w() if post else None,
                      half(r, H, scale=0.1) if post else None, w() if gate else None, 0.5, kind,
                      1e-5, offset)


@pytest.mark.parametrize("T", [1, 7, 130])
@pytest.mark.parametrize("kind,post,gate,offset", [(M.MOE_NORM_RMS, False, False, False),
                                                   (M.MOE_NORM_RMS, True, True, True),
                                                   (M.MOE_NORM_LAYER, True, False, False)])
def test_stack_with_norms(T, kind, post, gate, offset):
    say("stack with norms T=%d" % T)
    H, I, E, k = 256, 128, 8, 2
    r = np.random.default_rng(T)
    layers = [layer(r, H, I, E, k, None if l != 1 else ScoreRouting(),
                    norms(r, H, kind, post, gate, offset), l == 1) for l in range(3)]
    bufs = [lay.buffers(T) for lay in layers]
    acts = [half(r, T, H)] + [torch.empty((T, H), dtype=torch.float16, device=DEV) for _ in layers]
    assert stack_forward(layers, bufs, acts) is acts[3]
    torch.cuda.synchronize()
    c = dict(kind="rms" if kind == M.MOE_NORM_RMS else "layer", post=post, scale=0.5, eps=1e-5,
             offset=offset)
    v = lambda t: None if t is None else t.cpu().double()  # noqa: E731
    start = dict(c, post=False, scale=1.0)
    t0 = dict(y=None, residual=v(acts[0]), gate=None, pre_w=v(layers[0].norms.pre_w),
              pre_b=v(layers[0].norms.pre_b))
    n, size = B.block_norm_ref(start, t0)[1], B.block_norm_sizes(start, t0)[1]
    for l, lay in enumerate(layers):
        got = v(bufs[l].normed)
        assert ((got - n).abs() <= 2.0 ** -11 * n.abs() + STEPS * B.U * size + 1e-7).all()
        # the block itself: the layer's own calls on the normed rows, the same bits
        b = lay.buffers(T)
        out = lay.forward(bufs[l].normed, b)
        torch.cuda.synchronize()
        assert torch.equal(out, bufs[l].out) and torch.equal(b.topk_idx, bufs[l].topk_idx)
        nx = layers[l + 1].norms if l < 2 else lay.norms
        t = dict(y=v(out), residual=v(acts[l]), gate=v(lay.norms.gate),
                 post_w=v(lay.norms.post_w), post_b=v(lay.norms.post_b), pre_w=v(nx.pre_w),
                 pre_b=v(nx.pre_b))
        h, n = B.block_norm_ref(c, t)
        sh, size = B.block_norm_sizes(c, t)
        got = v(acts[l + 1])
        assert ((got - h).abs() <= 2.0 ** -11 * h.abs() + STEPS * B.U * sh + 1e-7).all()


@pytest.mark.parametrize("T", [1, 2, 9, 70, 300])
@pytest.mark.parametrize("H,E", [(384, 24), (2560, 60)])
def test_router_of_other_widths(T, H, E):
    """Score-routed FP8 layers whose width the pinned-order router does not take."""
    say("router H=%d T=%d" % (H, T))
    r = np.random.default_rng(T + H)
    lay = layer(r, H, 64, E, 4, ScoreRouting(), None, True)
    b, x = lay.buffers(T), half(r, T, H)
    out = lay.forward(x, b, residual=x)
    torch.cuda.synchronize()
    xv, wv = x.cpu().double(), lay.router.cpu().double()
    want = xv @ wv.t() + lay.bias.cpu().double()
    size = xv.abs() @ wv.abs().t() + lay.bias.cpu().double().abs()
    assert ((b.logits.cpu().double() - want).abs() <= (H + 16) * B.U * size).all()
    idx, w = R.select(b.logits.cpu().numpy(), np.zeros(E), 4, "sigmoid", 1, 1, False, False, 1.0)
    assert np.array_equal(b.topk_idx.cpu().numpy(), idx)
    assert torch.isfinite(out).all()


def l2(got, want):
    got, want = got.cpu().double(), want.double()
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("H,E,k,routing,T", [
    (256, 16, 4, None, 200), (2048, 60, 4, "softmax", 333), (384, 24, 3, "sigmoid", 65),
    (1024, 64, 8, "sigmoid", 1), (512, 8, 2, None, 40)])
def test_router_training_step(H, E, k, routing, T):
    """Norm, router, selection, balance loss and back to the rows before the norm,
    against the chain's definition in 64 bits (the normed rows and the choices as the
    kernels formed them).  Gradients pass two roundings to fp16 (the logits' gradient,
    the normed rows'), each of an L2 below 2^-11 / sqrt(3), and fp32 sums."""
    say("router training step H=%d T=%d" % (H, T))
    r = np.random.default_rng(H + T)
    rt = None if routing is None else ScoreRouting(
        M.MOE_SCORE_SOFTMAX if routing == "softmax" else M.MOE_SCORE_SIGMOID)
    nm = norms(r, H, M.MOE_NORM_RMS, False, False)
    lay = layer(r, H, 64, E, k, rt, nm, True)
    b, g = lay.buffers(T), lay.balance_buffers(T)
    h = half(r, T, H)
    mask = torch.from_numpy((r.random(T) < 0.8).astype(np.uint8)).to(DEV)
    mask[0] = 1
    scale = torch.full((1,), 65536.0, device=DEV)
    coef, zcoef = 0.02, 0.001

    def step():
        M.moe_block_norm(None, 0, h, H, None, 0, 1.0, None, None, nm.pre_w, nm.pre_b,
                         M.MOE_DTYPE_F16, nm.w_dtype, nm.kind, 0, nm.eps, T, H, None, 0, b.normed, H)
        lay.route_permute(b.normed, b)
        lay.balance(b.normed, b, g, coef, zcoef, mask, scale)
        lay.router_backward(b.normed, g)
        dn = g.dx.half()
        out = [torch.empty_like(h), torch.empty(H, device=DEV), torch.empty(H, device=DEV)]
        nb = M.moe_block_norm_backward_workspace_bytes(T, H)
        ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
        M.moe_block_norm_backward(None, 0, dn, H, None, 0, h, H, None, 0, 1.0, None, None,
                                  nm.pre_w, M.MOE_DTYPE_F16, nm.w_dtype, nm.kind, 0, nm.eps, T, H,
                                  None, out[0], None, None, None, out[1], out[2], ws, nb)
        return out
    dh, dw, db = step()
    torch.cuda.synchronize()
    n16 = b.normed.cpu().double()
    wr, br = lay.router.cpu().double(), lay.bias.cpu().double()
    logits = n16 @ wr.t() + br
    score = M.MOE_SCORE_SOFTMAX if rt is None else rt.score
    counts, mean, losses, dl = B.balance_ref(logits, b.topk_idx.cpu(), mask.cpu(), E, score, coef,
                                             zcoef, 65536.0)
    assert torch.equal(g.counts.cpu().long(), counts)
    assert np.allclose(g.losses.cpu().numpy(), losses, rtol=1e-5)
    assert l2(g.mean_prob, mean) < 1e-5
    one = 2.0 ** -11 / 3 ** 0.5
    assert l2(g.dlogits, dl) < 1.2 * one + 1e-5
    room = 1.2 * one + 1e-5
    assert l2(g.d_router, dl.t() @ n16) < room * 3 and l2(g.d_bias, dl.sum(0)) < room * 3
    assert l2(g.dx, dl @ wr) < room * 3
    hv = h.cpu().double().requires_grad_(True)
    pw = nm.pre_w.cpu().double().requires_grad_(True)
    n = B.norm_ref(hv, pw, nm.pre_b.cpu().double(), "rms", nm.eps, False)
    want = torch.autograd.grad(n, [hv, pw], dl @ wr)
    assert l2(dh, want[0]) < room * 4 and l2(dw, want[1]) < room * 4
    assert l2(db, (dl @ wr).sum(0)) < room * 4
    # captured: every replay on new rows gives the eager step's bits
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        h.copy_(half(r, T, H))
        eager = [t.clone() for t in step()] + [g.losses.clone(), g.d_router.clone(), g.d_bias.clone()]
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(outs + [g.losses, g.d_router, g.d_bias], eager):
            assert torch.equal(a, e)
