"""Whole layers with score routing and FP8 experts (MoELayer), against 64-bit
references of the same chain: logits -> selection -> grouping -> experts ->
combine; and stacks that mix them with W4A16 layers."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
from int4_weight_only_router_amd.layer import (MoELayer, ScoreRouting, blob_table, load_experts,
                                               load_experts_fp8, stack_forward)
from tests import fp8_util as R
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def _layer(r, H, I, E, k, routing=None, fmt=M.MOE_FMT_FP8, renorm=False, shared=None):
    w = [tuple(r.normal(0, 0.02, s).astype(np.float32) for s in ((I, H), (I, H), (H, I)))
         for _ in range(E)]
    router = torch.from_numpy(r.normal(0, 0.05, (E, H)).astype(np.float16)).to(DEV)
    if fmt == M.MOE_FMT_FP8:
        blobs, g = load_experts_fp8(w, H, I, DEV), 0
    else:
        blobs, g = load_experts(w, H, I, 64, DEV)[0], 64
    lay = MoELayer(H, I, E, k, g, router, blob_table(blobs), None, shared, renorm=renorm,
                   device=DEV, fmt=fmt, routing=routing)
    lay._blobs = blobs
    return lay


def _values(lay):
    off, _ = M.moe_fp8_blob_layout(lay.H, lay.I)
    out = []
    for e in range(lay.E):
        each = []
        for j, (n, c) in enumerate(((lay.I, lay.H), (lay.I, lay.H), (lay.H, lay.I))):
            ns = R.blocks(n) * R.blocks(c)
            q = lay._blobs[e, off[j]:off[j] + n * c]
            s = lay._blobs[e, off[3 + j]:off[3 + j] + 4 * ns].contiguous().view(torch.float32)
            each.append((R.codes(q).reshape(n, c), s.cpu().numpy().reshape(R.blocks(n), -1)))
        out.append(each)
    return out


@pytest.mark.parametrize("T", [1, 3, 20, 150])
@pytest.mark.parametrize("shared", [False, True])
def test_layer(T, shared):
    say("fp8 layer T=%d shared=%d" % (T, shared))
    H, I, E, k = 256, 192, 24, 4
    r = np.random.default_rng(T)
    bias = r.normal(0, 0.1, E).astype(np.float32)
    rt = ScoreRouting(M.MOE_SCORE_SIGMOID, torch.from_numpy(bias).to(DEV), 4, 2, True, 2.5)
    sh = tuple(torch.from_numpy(r.normal(0, 0.02, s).astype(np.float16)).to(DEV)
               for s in ((128, H), (128, H), (H, 128))) if shared else None
    lay = _layer(r, H, I, E, k, rt, renorm=True, shared=sh)
    b = lay.buffers(T)
    x = torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV)
    out = lay.forward(x, b, residual=x)
    torch.cuda.synchronize()
    idx, w = R.select(b.logits.cpu().numpy(), bias, k, "sigmoid", 4, 2, True, True, 2.5)
    assert np.array_equal(b.topk_idx.cpu().numpy(), idx)
    counts, offsets, perm, inv = R.grouping(idx, E)
    assert np.array_equal(b.perm.cpu().numpy(), perm)
    vals, xf = _values(lay), x.float().cpu().numpy()
    y, dy = np.zeros((T * k, H)), np.zeros((T * k, H))
    for e in range(E):
        s = slice(offsets[e], offsets[e + 1])
        if counts[e]:
            y[s], dy[s] = R.experts_row(xf[perm[s] // k], *vals[e])
    dy = dy + 2.0 ** -11 * (np.abs(y) + dy) + 2.0 ** -25      # y is rounded to fp16
    take = inv.reshape(T, k)
    ref = (w[:, :, None] * y[take]).sum(1) + xf
    tol = (w[:, :, None] * dy[take]).sum(1)
    mag = (w[:, :, None] * np.abs(y[take])).sum(1) + np.abs(xf)
    if shared:
        s = b.shared_out.double().cpu().numpy()     # the fp16 path has its own tests
        ref, mag = ref + s, mag + np.abs(s)
    # weights carry 2 roundings; k + 2 additions in fp32; one fp16 rounding
    tol = tol + (k + 4) * 2 * R.U32 * mag
    tol = tol + 2.0 ** -11 * (np.abs(ref) + tol)
    off = np.abs(out.double().cpu().numpy() - ref) - tol
    assert np.all(off <= 0), "off by %g over the bound" % off.max()


@pytest.mark.parametrize("T", [1, 2, 40])
def test_stack_mixes_formats(T):
    """INT4 and FP8 layers, softmax and score routing in one stack: the fused
    forms give the bits of layer-by-layer calls."""
    say("mixed stack T=%d" % T)
    H, I, E, k = 256, 128, 16, 2
    r = np.random.default_rng(9)
    sig = ScoreRouting(M.MOE_SCORE_SIGMOID, None, 4, 2, False, 1.0)
    layers = [_layer(r, H, I, E, k, None, M.MOE_FMT_SYM), _layer(r, H, I, E, k),
              _layer(r, H, I, E, k, sig), _layer(r, H, I, E, k, sig, M.MOE_FMT_SYM),
              _layer(r, H, I, E, k, None, M.MOE_FMT_SYM), _layer(r, H, I, E, k, None, M.MOE_FMT_SYM)]
    x = torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV)
    parts = torch.empty(M.moe_logit_partials_bytes() // 4, device=DEV)
    runs = []
    for fuse, p in ((False, None), (True, None), (True, parts)):
        bufs = [lay.buffers(T) for lay in layers]
        acts = [x] + [torch.full((T, H), -7.0, dtype=torch.float16, device=DEV) for _ in layers]
        stack_forward(layers, bufs, acts, fuse=fuse, parts=p)
        torch.cuda.synchronize()
        runs.append(acts)
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)
    assert bool(runs[0][-1].isfinite().all())


def test_refusals():
    r = np.random.default_rng(0)
    lay = _layer(r, 256, 64, 4, 2)
    b = lay.buffers(1)
    with pytest.raises(ValueError):
        lay.pool_args(b, torch.empty(2, dtype=torch.int32))
    sig = _layer(r, 256, 64, 4, 2, ScoreRouting())
    with pytest.raises(ValueError):
        lay.combine_route_next(b, sig, sig.buffers(1))
    assert not lay.route_from_partials_ok(b) and not lay.split_route_ok(b, sig)


@pytest.mark.parametrize("T", [1, 30])
def test_layer_captured(T):
    """A captured layer over several replays, eager layers on their own buffers between."""
    say("fp8 layer graph T=%d" % T)
    H, I, E, k = 512, 128, 32, 4
    r = np.random.default_rng(T)
    lay = _layer(r, H, I, E, k, ScoreRouting(M.MOE_SCORE_SIGMOID, None, 8, 3, True, 1.5))
    xs = [torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV) for _ in range(4)]
    b, eb = lay.buffers(T), lay.buffers(T)
    xb = xs[0].clone()
    lay.forward(xb, b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lay.forward(xb, b)
    for x in xs[1:] + xs[:1]:
        xb.copy_(x)
        g.replay()
        want = lay.forward(x, eb)
        torch.cuda.synchronize()
        assert torch.equal(b.out, want)


def test_load_on_another_stream():
    """Loading on a side stream, by object or address, gives the same blobs."""
    H, I = 1024, 512
    r = np.random.default_rng(3)
    w = [tuple(r.normal(0, 0.02, s).astype(np.float32) for s in ((I, H), (I, H), (H, I)))
         for _ in range(4)]
    want = load_experts_fp8(w, H, I, DEV)
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = load_experts_fp8(w, H, I, DEV, s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
