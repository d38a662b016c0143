"""FP8 experts and layers on the GPU within the L2 bound that wrong results do
not fit in (fp8_strict), at the sizes of real layers and at ragged ones."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
from int4_weight_only_router_amd.layer import ScoreRouting
from tests import fp8_strict as S
from tests import fp8_util as R
from tests import test_gpu_fp8 as G
from tests import test_gpu_fp8_layer as L
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
DECODE, BATCHED = M.MOE_REGIME_DECODE, M.MOE_REGIME_BATCHED


def _rows_within(y, x, perm, offsets, vals, k, runs):
    """Every routed row of y [rows, H] (fp64) within its bound."""
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a < b:
            ref, allowed = S.experts_l2(x[perm[a:b] // k], *vals[e], runs)
            err = np.linalg.norm(y[a:b] - ref, axis=1)
            assert np.all(err <= allowed), "expert %d: %g of its bound" % (e, (err / allowed).max())


@pytest.mark.parametrize("T,H,I,E,k,regime", [
    (1, 2048, 1024, 16, 8, DECODE), (1, 2048, 1024, 16, 8, BATCHED), (11, 2048, 1408, 6, 2, DECODE),
    (11, 2048, 1408, 6, 2, BATCHED), (70, 2048, 512, 6, 2, BATCHED), (70, 2048, 512, 6, 2, DECODE),
    (400, 2048, 1024, 4, 1, BATCHED), (300, 512, 448, 3, 1, BATCHED), (5, 256, 192, 8, 2, DECODE),
    (100, 320, 192, 4, 2, BATCHED), (9, 64, 8192, 2, 2, DECODE), (3, 8192, 64, 2, 1, BATCHED)])
def test_experts(T, H, I, E, k, regime):
    say("experts strict T=%d H=%d I=%d E=%d k=%d regime=%d" % (T, H, I, E, k, regime))
    r = np.random.default_rng(T * 13 + H + I)
    dev, vals, table = G._blobs(r, E, H, I)
    x = torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV)
    perm, offsets = G._grouping(np.argsort(r.normal(0, 1, (T, E)), 1)[:, :k], E)
    y = G._ffn(x, perm, offsets, table, T, H, I, E, k, regime)
    _rows_within(y.double().cpu().numpy(), x.float().cpu().numpy(), perm.cpu().numpy(),
                 offsets.cpu().numpy(), vals, k, regime == BATCHED)


@pytest.mark.parametrize("T", [1, 40])
def test_layer(T):
    """The layer's rows of y within their bound, and out combined from them."""
    say("fp8 layer strict T=%d" % T)
    H, I, E, k = 2048, 512, 12, 3
    r = np.random.default_rng(T)
    lay = L._layer(r, H, I, E, k, ScoreRouting(M.MOE_SCORE_SIGMOID, None, 4, 2, True, 2.5),
                   renorm=True)
    b = lay.buffers(T)
    x = torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV)
    out = lay.forward(x, b, residual=x)
    torch.cuda.synchronize()
    y = b.y[0, :T * k].double().cpu().numpy()
    _rows_within(y, x.float().cpu().numpy(), b.perm.cpu().numpy(), b.offsets.cpu().numpy(),
                 L._values(lay), k, b.regime & 0xFF == BATCHED)
    w = b.topk_w.double().cpu().numpy()
    each = w[:, :, None] * y[b.inv_perm.cpu().numpy().reshape(T, k)]
    ref, mag = each.sum(1) + x.double().cpu().numpy(), np.abs(each).sum(1) + x.double().abs().cpu().numpy()
    # k + 2 additions in fp32, each at most a step; one fp16 rounding
    tol = (k + 2) * 2 * R.U32 * mag
    tol = tol + 2.0 ** -11 * (np.abs(ref) + tol) + 2.0 ** -25
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)


def _cancelling(H, I):
    """An expert whose h is one value in every column (gate and up rows are
    alike), so that y[n] is h times the sum of down's row n: row 0 is ones, every
    other row's runs of eight cancel but for small products far below the run's
    largest.  Returns its blob and the sums."""
    off, total = M.moe_fp8_blob_layout(H, I)
    r = np.random.default_rng(I)
    blob = np.zeros(total, np.uint8)
    ones = torch.ones(1).to(G.F8).view(torch.uint8).numpy()[0]
    blob[off[0]:off[0] + 2 * I * H] = ones                 # (the sections follow each other)
    wd = np.zeros((H, I), np.float32)
    wd[0] = 1.0
    for n in range(1, H):
        runs = np.zeros((I // 8, 8), np.float32)
        runs[:, 0], runs[:, 1] = 256, -256
        runs[:, 2:] = R.e4m3(np.exp2(r.uniform(-8, -4, (I // 8, 6))))
        wd[n] = runs.reshape(-1)
    assert off[1] - off[0] == I * H
    blob[off[2]:off[2] + H * I] = torch.from_numpy(wd).to(G.F8).view(torch.uint8).numpy().reshape(-1)
    nb = R.blocks(H) * R.blocks(I)
    for j, s in ((3, 2.0 ** -14), (4, 1.0), (5, 1.0)):
        blob[off[j]:off[j] + 4 * nb] = np.full(nb, s, np.float32).view(np.uint8)
    return torch.from_numpy(blob).to(DEV), wd.astype(np.float64).sum(1)


def _cancelled(T, H, I, regime):
    """(y of T equal tokens, what it should be, its fp32 bound)."""
    blob, sums = _cancelling(H, I)
    table = torch.tensor([blob.data_ptr()], device=DEV)
    x = torch.ones((T, H), dtype=torch.float16, device=DEV)
    perm, offsets = G._grouping(np.zeros((T, 1), np.int64), 1)
    y = G._ffn(x, perm, offsets, table, T, H, I, 1, 1, regime)[:T].double().cpu().numpy()
    # g = H 2^-14, u = H: sums of equal powers of two, exact; h = silu(g) u; its
    # code and scale are the same in every column, so y[n] = (code scale) sums[n]
    g = H * 2.0 ** -14
    h = g / (1.0 + np.exp(-g)) * H
    s = float(R.scale_of(np.float32([h]), True)[0])
    code = float(R.e4m3(h / s)) * s
    assert float(R.e4m3(h / s * (1 - 1e-4))) == float(R.e4m3(h / s * (1 + 1e-4)))
    bound = (256 + R.blocks(I) + 4) * R.U32 * (512 * I / 8 + 6 * I / 8 * 2.0 ** -4) * code
    ref = code * sums
    return y, ref, bound + 2.0 ** -11 * (np.abs(ref) + bound) + 2.0 ** -25


@pytest.mark.parametrize("T", [1, 3, 16])
def test_decode_sums_in_fp32(T):
    """DECODE's down keeps small products beside large ones that cancel."""
    say("experts cancelling T=%d" % T)
    y, ref, tol = _cancelled(T, 256, 128, DECODE)
    assert np.all(np.abs(y - ref) <= tol)
    assert np.abs(ref[1:]).min() > 4 * tol[1:].max()   # the bound tells the sums from zero
