"""Expert selection from logits (moe_route_select, moe_route_select_permute)
and the public router logits, on the GPU against 64-bit references: indices
and groupings equal, weights within two fp32 roundings."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
import moe_inputs as MI
from tests import fp8_util as R
from tests.gpu_util import DEV, f16, say

pytestmark = pytest.mark.gpu
TYPES = {"f32": (torch.float32, M.MOE_DTYPE_F32), "f16": (torch.float16, M.MOE_DTYPE_F16),
         "bf16": (torch.bfloat16, M.MOE_DTYPE_BF16)}


def _run(l, bias, k, score, n_group, keep, top2, renorm, scale, dtype="f32", ld=None, fused=True,
         stream=None):
    T, E = l.shape
    tt, dt = TYPES[dtype]
    ld = E if ld is None else ld
    buf = torch.full((max(T, 1), ld), float("nan"), dtype=tt, device=DEV)
    buf[:T, :E] = torch.as_tensor(l).to(tt).to(DEV)
    b = None if bias is None else torch.as_tensor(bias, dtype=torch.float32).to(DEV)
    n = T * k
    i32 = lambda m: torch.full((m + 3,), -7, dtype=torch.int32, device=DEV)   # noqa: E731
    idx, counts, offsets, perm, inv = i32(n), i32(E), i32(E + 1), i32(n), i32(n)
    w = torch.full((n + 3,), -7.0, device=DEV)
    flags = (M.MOE_RENORM if renorm else 0) | (M.MOE_GROUP_TOP2 if top2 else 0)
    sc = M.MOE_SCORE_SOFTMAX if score == "softmax" else M.MOE_SCORE_SIGMOID
    if fused:
        nws = M.moe_route_select_workspace_bytes(T, k, E)
        ws = torch.full((max(nws, 1),), 0xAB, dtype=torch.uint8, device=DEV)
        M.moe_route_select_permute(buf, dt, ld, b, T, E, k, sc, n_group, keep, flags, scale, idx,
                                   w, counts, offsets, perm, inv, ws, nws, stream)
    else:
        M.moe_route_select(buf, dt, ld, b, T, E, k, sc, n_group, keep, flags, scale, idx, w,
                           stream)
    torch.cuda.synchronize()
    out = [t.cpu().numpy() for t in (idx, w, counts, offsets, perm, inv)]
    for t, m in zip(out, (n, n, E, E + 1, n, n)):
        assert (t[m if fused or t is out[0] or t is out[1] else 0:] == -7).all()   # nothing behind
    idx, w, counts, offsets, perm, inv = (t[:-3] for t in out)
    return idx.reshape(T, k), w.reshape(T, k), counts, offsets, perm, inv, \
        buf[:T, :E].float().cpu().numpy()


def _check(l, bias, k, score, n_group=1, keep=1, top2=False, renorm=False, scale=1.0, **kw):
    idx, w, counts, offsets, perm, inv, used = _run(l, bias, k, score, n_group, keep, top2,
                                                    renorm, scale, **kw)
    ri, rw = R.select(used, bias, k, score, n_group, keep, top2, renorm, scale)
    assert np.array_equal(idx, ri)
    assert np.all(np.abs(w - rw) <= 2 * R.U32 * np.abs(rw) + 2.0 ** -149)
    if kw.get("fused", True):
        for a, b in zip((counts, offsets, perm, inv), R.grouping(ri, l.shape[1])):
            assert np.array_equal(a, b)


CASES = [   # T, E, k, groups, keep, top2
    (1, 1, 1, 1, 1, False), (1, 8, 2, 1, 1, False), (1, 64, 8, 1, 1, False),
    (3, 60, 4, 6, 3, False), (16, 512, 10, 8, 4, True), (17, 512, 10, 8, 4, True),
    (5, 1024, 16, 64, 9, True), (33, 1000, 16, 8, 3, True), (9, 65, 16, 5, 2, True),
    (130, 256, 8, 8, 4, True), (67, 96, 6, 4, 4, False), (2, 129, 1, 3, 1, True),
    (1025, 60, 4, 60, 4, False), (12, 640, 7, 10, 1, False), (8, 1024, 16, 1, 1, False),
    (1, 1024, 16, 64, 2, True), (1, 130, 5, 2, 1, False), (9, 1000, 3, 8, 2, True),
    (8192, 64, 2, 8, 3, True), (8193, 16, 2, 1, 1, False), (40, 768, 9, 3, 2, True)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,keep,top2", CASES)
def test_select(T, E, k, G, keep, top2, score):
    say("select T=%d E=%d k=%d groups=%d/%d %s" % (T, E, k, keep, G, score))
    r = np.random.default_rng(T * 1000 + E)
    l = r.normal(0, 0.9, (T, E)).astype(np.float32)
    b = r.normal(0, 0.05, E).astype(np.float32)
    _check(l, b, k, score, G, keep, top2, True, 2.5)
    _check(l, None, k, score, G, keep, top2, False, 1.0, fused=False)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ld", [60, 61, 75])
def test_types_and_strides(dtype, ld):
    """Coarse types tie often; odd strides leave rows unaligned, with NaN between them."""
    say("select types %s ld=%d" % (dtype, ld))
    r = np.random.default_rng(7)
    l = np.round(r.normal(0, 0.9, (23, 60)) * 8) / 8
    _check(l.astype(np.float32), None, 5, "sigmoid", 4, 2, True, True, dtype=dtype, ld=ld)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks_ties_and_extremes(score):
    say("select masks %s" % score)
    r = np.random.default_rng(3)
    E = 96
    l = r.normal(0, 1, (14, E)).astype(np.float32)
    l[0] = -np.inf                                 # nothing left
    l[1] = np.nan
    l[2] = 0.25                                    # all tied
    l[3, 5:] = -np.inf                             # fewer live experts than k
    l[4, 17] = np.inf                              # counts as the largest finite value
    l[5] = np.finfo(np.float32).min                # the type's lowest value, not a mask
    l[6, ::2] = -np.inf
    l[7, 32:64] = -np.inf                          # a whole group masked
    l[8] = np.where(np.arange(E) % 3 == 0, 60.0, -60.0)   # saturated scores tie
    l[9, 1] = np.nan
    l[10] = -np.inf
    l[10, 95] = 1.0
    l[11] = 3.4e38
    l[12, :2] = np.inf
    l[13] = -0.0
    l[13, 50] = 0.0
    for G, keep, top2 in ((1, 1, False), (3, 2, True), (3, 1, False), (12, 5, True)):
        for renorm in (False, True):
            _check(l, None, 8, score, G, keep, top2, renorm)
            _check(l[:6], r.normal(0, 0.5, E).astype(np.float32), 8, score, G, keep, top2, renorm)


def test_many_ties_take_the_long_path():
    """More than 64 candidates at the bound: the k rounds of a wave-wide maximum."""
    say("select ties")
    l = np.zeros((3, 1024), np.float32)
    l[1, 500:] = 1.0
    l[2, ::5] = -1.0
    _check(l, None, 16, "softmax")
    _check(l, None, 16, "sigmoid", 4, 2, True, True)


def test_no_tokens_clears_the_grouping():
    idx, w, counts, offsets, perm, inv, _ = _run(np.zeros((0, 12), np.float32), None, 3,
                                                 "softmax", 1, 1, False, False, 1.0)
    assert not counts.any() and not offsets.any()


@pytest.mark.parametrize("T", [1, 4, 40])
def test_captured_and_replayed(T):
    """Replays of a captured call follow the logits that lie in its buffers then."""
    say("select graph T=%d" % T)
    E, k = 512, 10
    r = np.random.default_rng(T)
    buf = torch.zeros((T, E), device=DEV)
    i32 = lambda m: torch.zeros(m, dtype=torch.int32, device=DEV)   # noqa: E731
    idx, counts, offsets, perm, inv = i32(T * k), i32(E), i32(E + 1), i32(T * k), i32(T * k)
    w = torch.zeros(T * k, device=DEV)
    nws = M.moe_route_select_workspace_bytes(T, k, E)
    ws = torch.zeros(max(nws, 1), dtype=torch.uint8, device=DEV)

    def call():
        M.moe_route_select_permute(buf, M.MOE_DTYPE_F32, E, None, T, E, k, M.MOE_SCORE_SIGMOID, 8,
                                   4, M.MOE_GROUP_TOP2, 1.0, idx, w, counts, offsets, perm, inv,
                                   ws, nws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        l = r.normal(0, 1, (T, E)).astype(np.float32)
        buf.copy_(torch.from_numpy(l))
        g.replay()
        torch.cuda.synchronize()
        ri, _ = R.select(l, None, k, "sigmoid", 8, 4, True, False, 1.0)
        assert np.array_equal(idx.cpu().numpy().reshape(T, k), ri)
        assert np.array_equal(perm.cpu().numpy(), R.grouping(ri, E)[2])


@pytest.mark.parametrize("cfg,T", [(MI.TINY, 1), (MI.TINY, 3), (MI.OLMOE_DECODE, 1),
                                   (MI.OLMOE_DECODE, 4), (MI.OLMOE_DECODE, 5), (MI.E512, 2),
                                   (MI.E512, 70)], ids=lambda v: getattr(v, "name", str(v)))
def test_logits_select_equals_route(cfg, T):
    """moe_router_logits + moe_route_select in the softmax form without groups
    chooses what moe_route chooses, and the logits are 64-bit sums up to fp32."""
    say("router logits %s T=%d" % (cfg.name, T))
    x, wr = MI.gen_x(cfg, T), MI.gen_router(cfg)
    b = MI.zipf_bias(cfg)
    bias = None if b is None else torch.from_numpy(b).to(DEV)
    lg = torch.empty((T, cfg.E), device=DEV)
    M.moe_router_logits(f16(x), f16(wr), bias, T, cfg.H, cfg.E, lg)
    mk = lambda: (torch.empty((T, cfg.k), dtype=torch.int32, device=DEV),   # noqa: E731
                  torch.empty((T, cfg.k), device=DEV))
    (i0, w0), (i1, w1) = mk(), mk()
    M.moe_route_select(lg, M.MOE_DTYPE_F32, cfg.E, None, T, cfg.E, cfg.k, M.MOE_SCORE_SOFTMAX, 1,
                       1, 0, 1.0, i0, w0)
    nws = M.moe_route_workspace_bytes(T, cfg.E)
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=DEV)
    M.moe_route(f16(x), f16(wr), bias, T, cfg.H, cfg.E, cfg.k, 0, i1, w1, ws, nws)
    torch.cuda.synchronize()
    assert torch.equal(i0, i1)
    assert float((w0 - w1).abs().max()) <= 1e-6     # moe_route's softmax is in fp32
    x64, w64 = x.astype(np.float64), wr.astype(np.float64)
    ref = x64 @ w64.T + (0 if b is None else b)
    # at most 32 additions in a lane, 6 across lanes, one for the bias
    bound = 40 * R.U32 * (np.abs(x64) @ np.abs(w64).T + (0 if b is None else np.abs(b)))
    assert np.all(np.abs(lg.cpu().numpy() - ref) <= bound)
