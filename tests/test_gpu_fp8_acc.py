"""MOE_ACC_F32: 16-bit outputs of FP8 products and experts with the accuracy of
fp32 sums at every size, on products that cancel and on random ones."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
from int4_weight_only_router_amd.layer import ScoreRouting
from tests import fp8_util as R
from tests import test_gpu_fp8 as G
from tests import test_gpu_fp8_layer as L
from tests import test_gpu_fp8_strict as S
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
ACC = M.MOE_ACC_F32


def _gemm(xv, xs, wv, ws, dtype, flag=ACC, ldo=None):
    (m, k), n = xv.shape, wv.shape[0]
    codes = lambda v: torch.from_numpy(v.astype(np.float32)).to(G.F8).view(torch.uint8).to(DEV)  # noqa: E731
    scale = lambda s: torch.from_numpy(s).to(DEV)   # noqa: E731
    tt, dt = G.TYPES[dtype]
    out = torch.full((m + 1, ldo or n), -7.0, dtype=tt, device=DEV)
    M.moe_gemm_fp8(codes(xv), k, scale(xs), codes(wv), k, scale(ws), m, n, k, out, dt | flag,
                   ldo or n)
    torch.cuda.synchronize()
    assert bool((out[m] == -7.0).all()) and bool((out[:m, n:] == -7.0).all())
    return out[:m, :n].double().cpu().numpy()


def _rounded(y, bound, dtype):
    half = R.HALF_STEP[G.TYPES[dtype][0]]
    return bound + half * (np.abs(y) + bound) + (2.0 ** -25 if dtype == "f16" else 0.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k,ldo", [
    (1, 33, 48, None), (17, 130, 144, 131), (333, 1408, 2000, None), (1600, 4001, 144, 4003),
    (1531, 4117, 400, None), (130, 24700, 144, None), (1000, 1500, 272, None),
    (700, 5000, 144, None), (2500, 5000, 80, 5008), (2000, 9000, 48, None)])
def test_product(m, n, k, ldo, dtype):
    say("product fp32 sums %dx%dx%d %s" % (m, n, k, dtype))
    r = np.random.default_rng(m + n + k)
    xv, wv = (R.e4m3(np.clip(r.normal(0, 60, s), -448, 448)) for s in ((m, k), (n, k)))
    xs = np.exp(r.normal(-6, 1, (m, R.blocks(k)))).astype(np.float32)
    ws = np.exp(r.normal(-6, 1, (R.blocks(n), R.blocks(k)))).astype(np.float32)
    y, bound = R.product(xv, xs, wv, ws)
    off = np.abs(_gemm(xv, xs, wv, ws, dtype, ldo=ldo) - y) - _rounded(y, bound, dtype)
    assert np.all(off <= 0), "off by %g over the bound" % off.max()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n", [(1, 64), (40, 64), (300, 5632), (600, 5632), (1024, 5632),
                                 (4096, 1536)])
def test_products_that_cancel(m, n, dtype):
    """Runs of eight whose large products cancel and whose others lie 13 bits
    below them: with the flag they count in a row of any batch; without it they
    may be lost up to the stated bound, and no further."""
    say("product cancelling %dx%d %s" % (m, n, dtype))
    k = 256
    r = np.random.default_rng(n)
    wv = R.e4m3(np.exp2(r.uniform(-8, -4, (n, k))))
    wv[:, ::8], wv[:, 1::8] = 256, -256
    xv = np.ones((m, k))
    xv[::3] = 2
    xs, ws = np.ones((m, 2), np.float32), np.ones((R.blocks(n), 2), np.float32)
    y, bound = R.product(xv, xs, wv, ws)
    assert y.min() > 4 * bound.max()       # the bound tells the sums from zero
    assert np.all(np.abs(_gemm(xv, xs, wv, ws, dtype) - y) <= _rounded(y, bound, dtype))
    y, bound = R.product(xv, xs, wv, ws, runs=True)
    assert np.all(np.abs(_gemm(xv, xs, wv, ws, dtype, 0) - y) <= _rounded(y, bound, dtype))


@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (40, 256, 128), (200, 512, 320), (700, 256, 192)])
@pytest.mark.parametrize("regime", [M.MOE_REGIME_AUTO, M.MOE_REGIME_BATCHED])
def test_experts_that_cancel(T, H, I, regime):
    say("experts cancelling, fp32 sums T=%d H=%d I=%d regime=%d" % (T, H, I, regime))
    y, ref, tol = S._cancelled(T, H, I, regime | ACC)
    assert np.all(np.abs(y - ref) <= tol)
    assert np.abs(ref[1:]).min() > 4 * tol[1:].max()


@pytest.mark.parametrize("T,H,I,E,k,regime", [
    (11, 2048, 1408, 6, 2, M.MOE_REGIME_BATCHED), (11, 2048, 1408, 6, 2, M.MOE_REGIME_DECODE),
    (400, 2048, 1024, 4, 1, 0), (300, 512, 448, 3, 1, 0), (70, 2048, 512, 6, 2, 0)])
def test_experts(T, H, I, E, k, regime):
    say("experts fp32 sums T=%d H=%d I=%d" % (T, H, I))
    r = np.random.default_rng(T * 11 + H + I)
    dev, vals, table = G._blobs(r, E, H, I)
    x = torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV)
    perm, offsets = G._grouping(np.argsort(r.normal(0, 1, (T, E)), 1)[:, :k], E)
    y = G._ffn(x, perm, offsets, table, T, H, I, E, k, regime | ACC)
    S._rows_within(y.double().cpu().numpy(), x.float().cpu().numpy(), perm.cpu().numpy(),
                   offsets.cpu().numpy(), vals, k, False)
    assert bool((y[T * k:] == -7.0).all())


@pytest.mark.parametrize("T", [2, 60])
def test_layer(T):
    """A layer whose buffers carry the flag, captured and replayed."""
    say("fp8 layer fp32 sums T=%d" % T)
    H, I, E, k = 512, 256, 12, 3
    r = np.random.default_rng(T)
    lay = L._layer(r, H, I, E, k, ScoreRouting(M.MOE_SCORE_SIGMOID, None, 4, 2, True, 2.5))
    b, eb = (lay.buffers(T, M.MOE_REGIME_AUTO | ACC) for _ in range(2))
    assert b.regime & ACC
    xs = [torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV) for _ in range(3)]
    xb = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lay.forward(xb, b, residual=xb)
    for x in xs:
        xb.copy_(x)
        g.replay()
        want = lay.forward(x, eb, residual=x)
        torch.cuda.synchronize()
        assert torch.equal(b.out, want)
        S._rows_within(b.y[0, :T * k].double().cpu().numpy(), x.float().cpu().numpy(),
                       b.perm.cpu().numpy(), b.offsets.cpu().numpy(), L._values(lay), k, False)
