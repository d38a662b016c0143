"""moe_balance_loss against the 64-bit definition."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
from tests import block_util as R
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = R.U
SCORES = {"softmax": M.MOE_SCORE_SOFTMAX, "sigmoid": M.MOE_SCORE_SIGMOID}


def call(logits, idx, mask, k, score, coef, zcoef, up=None, gtype="f32", grad=True, pad=0,
         counts=None, E=None, stream=None, ws=None):
    T, E = logits.shape[0], logits.shape[1] if E is None else E
    o = [torch.full((E,), -7, dtype=torch.int32, device=DEV) if counts is None else counts,
         torch.full((E,), -7.0, device=DEV), torch.full((2,), -7.0, device=DEV)]
    dl = torch.full((T, E + pad), -7.0, dtype=R.TYPES[gtype][0], device=DEV) if grad else None
    nb = M.moe_balance_loss_workspace_bytes(T, E)
    if ws is None:
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=DEV)
    types = {t: c for t, c in R.TYPES.values()}
    M.moe_balance_loss(logits, types[logits.dtype], logits.shape[1], idx, mask, T, E, k,
                       SCORES[score], coef, zcoef, *o, up, dl, R.TYPES[gtype][1],
                       E + pad if grad else 0, ws, nb, stream)
    return o + ([dl] if grad else [])


def draw(T, E, k, masked=0.0, zipf=0.0, dtype="f32", seed=0, pad=0):
    g = torch.Generator().manual_seed(T + 31 * E + seed)
    l = 1.2 * torch.randn((T, E), generator=g)
    if zipf:
        l = l - zipf * torch.log(torch.randperm(E, generator=g).float() + 1)
    wide = torch.full((T, E + pad), 50.0, dtype=R.TYPES[dtype][0])
    wide[:, :E] = l.to(wide.dtype)
    idx = torch.sort(wide[:, :E].float(), dim=1, descending=True, stable=True)[1][:, :k].int()
    mask = None
    if masked:
        mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8) * 3   # any nonzero counts
    return wide, idx.contiguous(), mask


# A probability passes the exponentials (an argument of up to A is off by A half
# steps), a sum of E terms (16 a lane, 8 steps across the wave) and a quotient: below
# A + 40 half steps; a product sum p d another 24; the sum over the tokens one
# addition a row of a wave and the joins (16 partial sums of 4 waves at a time).
STEPS = 96


def check(got, l, idx, mask, E, k, score, coef, zcoef, up, gtype):
    counts, mean, losses, grad = R.balance_ref(l[:, :E].cpu(), idx, mask, E, SCORES[score], coef,
                                               zcoef, up)
    fl = l[:, :E].double()
    fl = fl[torch.isfinite(fl)]
    steps = STEPS + 2 * float(fl.max() - fl.min() if fl.numel() else 0.0)
    T = l.shape[0]
    assert torch.equal(got[0].cpu().long(), counts)
    sums = steps + T / 2048 + 80
    assert ((got[1].cpu().double() - mean).abs() <= sums * U * mean + 1e-30).all()
    want = torch.from_numpy(losses)
    assert ((got[2].cpu().double() - want).abs() <= 2 * sums * U * want.abs() + 1e-30).all()
    if len(got) < 4:
        return
    dt = R.TYPES[gtype][0]
    n = max(1, T if mask is None else int((mask != 0).sum()))
    total = max(1, int(counts.sum()))
    d = (counts.double() * E / total - 1.0).abs()
    out = got[3].cpu().double()
    on = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    ll = torch.where(torch.isnan(l[:, :E].cpu().double()), -np.inf, l[:, :E].cpu().double())
    ll = ll.clamp_max(torch.finfo(torch.float32).max)
    some = torch.isfinite(ll).any(dim=1) & on
    safe = torch.where(some[:, None], ll, torch.zeros_like(ll))
    soft = torch.softmax(safe, 1)
    logs = safe if score == "softmax" else torch.nn.functional.logsigmoid(safe)
    p = torch.softmax(logs, 1)
    size = coef / n * p * (d + (p * d).sum(1, keepdim=True)) \
        + abs(zcoef) * 2 / n * torch.logsumexp(safe, 1, keepdim=True).abs() * soft
    bound = up * 2 * steps * U * size + R.half_step(dt) * grad.abs() + R.tiny(dt)
    bad = ~((out[:, :E] - grad).abs() <= bound)
    assert not bad.any(), "%d off, worst %.3g of its bound" % (
        int(bad.sum()), float(((out[:, :E] - grad).abs() / bound).max()))
    assert (out[~some][:, :E] == 0).all()
    assert (out[:, E:] == -7.0).all()


CASES = [(1, 64, 8), (1, 1, 1), (2, 3, 3), (16, 64, 8), (63, 60, 4), (64, 1024, 16), (65, 1024, 16),
         (64, 17, 2), (65, 65, 3), (257, 512, 10), (300, 129, 5), (777, 60, 4), (1025, 256, 1),
         (2100, 384, 8)]


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("masked,zcoef,dtype,gtype,pad", [(0.0, 0.0, "f32", "f32", 0),
                                                          (0.3, 0.01, "f16", "bf16", 3),
                                                          (0.6, 0.002, "bf16", "f16", 1)])
@pytest.mark.parametrize("T,E,k", CASES)
def test_against_definition(T, E, k, masked, zcoef, dtype, gtype, pad, score):
    say("balance %dx%d %s" % (T, E, score))
    l, idx, mask = draw(T, E, k, masked, 1.1 if T % 2 else 0.0, dtype, pad=pad)
    up = torch.tensor([4096.0], device=DEV)
    dev = (l.to(DEV), idx.to(DEV), None if mask is None else mask.to(DEV))
    got = call(*dev, k, score, 0.01, zcoef, up, gtype, pad=pad, E=E)
    torch.cuda.synchronize()
    check(got, l, idx, mask, E, k, score, 0.01, zcoef, 4096.0, gtype)
    # without the gradient, and with the counts given: the same bits
    plain = call(*dev, k, score, 0.01, zcoef, grad=False, E=E)
    assert all(torch.equal(a, b) for a, b in zip(plain, got[:3]))
    given = call(dev[0], None, dev[2], k, score, 0.01, zcoef, up, gtype, pad=pad, E=E,
                 counts=got[0].clone())
    assert all(torch.equal(a, b) for a, b in zip(given, got))


@pytest.mark.parametrize("T,E,k,score", [(5000, 100, 4, "softmax"), (2500, 1000, 3, "sigmoid")])
def test_more_rows_than_waves(T, E, k, score):
    say("balance %dx%d %s" % (T, E, score))
    l, idx, mask = draw(T, E, k, 0.3, 1.1, "f16", pad=1)
    up = torch.tensor([64.0], device=DEV)
    got = call(l.to(DEV), idx.to(DEV), mask.to(DEV), k, score, 0.01, 0.01, up, "f16", pad=2, E=E)
    torch.cuda.synchronize()
    check(got, l, idx, mask, E, k, score, 0.01, 0.01, 64.0, "f16")


def test_given_counts_of_any_size():
    """Counts beyond what T tokens choose, such as those of many steps together."""
    l, idx, _ = draw(70, 60, 2)
    c = torch.randint(0, 1 << 30, (60,), generator=torch.Generator().manual_seed(2)).int()
    got = call(l.to(DEV), None, None, 2, "softmax", 0.5, 0.0, counts=c.to(DEV))
    f = c.double() / c.double().sum()
    p = torch.softmax(l.double(), 1)
    want = 0.5 * 60 * float((f * p.mean(0)).sum())
    assert abs(float(got[2][0]) - want) <= 4 * STEPS * U * want
    d = 60 * f - 1.0
    grad = 0.5 / 70 * p * (d - (p * d).sum(1, keepdim=True))
    size = 0.5 / 70 * p * (d.abs() + (p * d).abs().sum(1, keepdim=True))
    assert ((got[3].cpu().double() - grad).abs() <= 2 * (STEPS + 16) * U * size).all()


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("T", [9, 130])
def test_masked_experts_and_far_logits(T, score):
    E, k = 70, 4
    l, idx, mask = draw(T, E, k)
    l[0, 3], l[0, 69] = -np.inf, np.nan
    l[1, :] = -np.inf
    l[2, :] = np.nan
    l[3, 5] = np.inf            # counts as the largest finite value
    l[4, :] = -1000.0 + l[4]    # every sigmoid below fp32's range
    l[5, :] += 500.0
    l[6, :] = torch.finfo(torch.float32).min
    l[7, 1:] = -np.inf
    idx[8] = torch.tensor([-1, E, 3, 1 << 30], dtype=torch.int32)   # only one counts
    got = call(l.to(DEV), idx.to(DEV), None, k, score, 0.01, 0.0)
    torch.cuda.synchronize()
    check(got, l, idx, None, E, k, score, 0.01, 0.0, 1.0, "f32")
    keep = [i for i in range(T) if i not in (3, 6)]   # (their squares leave fp32's range)
    l, idx = l[keep].contiguous(), idx[keep].contiguous()
    got = call(l.to(DEV), idx.to(DEV), None, k, score, 0.01, 0.001)
    torch.cuda.synchronize()
    check(got, l, idx, None, E, k, score, 0.01, 0.001, 1.0, "f32")


@pytest.mark.parametrize("T", [5, 200])
def test_every_token_masked(T):
    l, idx, _ = draw(T, 40, 2)
    mask = torch.zeros(T, dtype=torch.uint8, device=DEV)
    got = call(l.to(DEV), idx.to(DEV), mask, 2, "softmax", 0.01, 0.1)
    assert all((t == 0).all() for t in got)


def test_masked_tokens_may_hold_anything():
    l, idx, mask = draw(100, 40, 2, masked=0.5)
    a = call(l.to(DEV), idx.to(DEV), mask.to(DEV), 2, "softmax", 0.01, 0.1)
    l[mask == 0], idx[mask == 0] = np.nan, -5
    b = call(l.to(DEV), idx.to(DEV), mask.to(DEV), 2, "softmax", 0.01, 0.1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_tokens():
    o = [torch.full((9,), 3, dtype=torch.int32, device=DEV), torch.ones(9, device=DEV),
         torch.ones(2, device=DEV)]
    M.moe_balance_loss(None, M.MOE_DTYPE_F32, 9, None, None, 0, 9, 2, 0, 1.0, 1.0, *o)
    assert all((t == 0).all() for t in o)


def test_optional_outputs():
    l, idx, _ = draw(90, 33, 3)
    full = call(l.to(DEV), idx.to(DEV), None, 3, "softmax", 0.01, 0.1)
    nb = M.moe_balance_loss_workspace_bytes(90, 33)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    counts = torch.empty(33, dtype=torch.int32, device=DEV)
    M.moe_balance_loss(l.to(DEV), M.MOE_DTYPE_F32, 33, idx.to(DEV), None, 90, 33, 3, 0, 0.01, 0.1,
                       counts, None, None, ws=ws, ws_bytes=nb)
    assert torch.equal(counts, full[0])


@pytest.mark.parametrize("score", list(SCORES))
def test_gradient_against_differences(score):
    """Along random directions, against central differences of the 64-bit losses with
    the counts held; the step's error is bounded by what half the step changes."""
    T, E, k = 30, 20, 3
    l, idx, _ = draw(T, E, k)
    coef, zcoef = 0.5, 0.05
    g = call(l.to(DEV), idx.to(DEV), None, k, score, coef, zcoef)[3].cpu().double()
    gen = torch.Generator().manual_seed(2)

    def loss(x):
        return float(R.balance_ref(x, idx, None, E, SCORES[score], coef, zcoef)[2].sum())
    for _ in range(3):
        e = torch.randn((T, E), generator=gen, dtype=torch.float64)
        slope = [(loss(l.double() + h * e) - loss(l.double() - h * e)) / (2 * h)
                 for h in (1e-4, 5e-5)]
        room = abs(slope[0] - slope[1]) + 1e-9 + 4 * STEPS * U * float((g * e).abs().sum())
        assert abs(float((g * e).sum()) - slope[1]) <= room


def test_far_rows():
    """Logits and gradients whose offsets pass 2^32 bytes."""
    E, stride, T = 64, 3 << 29, 3
    l, idx, _ = draw(T, E, 2)
    far = torch.empty(2 * stride + E, device=DEV)
    rows = far.as_strided((T, E), (stride, 1))
    rows.copy_(l)
    want = call(l.to(DEV), idx.to(DEV), None, 2, "softmax", 0.01, 0.1)
    out = torch.empty(2 * stride + E, dtype=torch.float16, device=DEV)
    o = [torch.empty_like(t) for t in want[:3]]
    M.moe_balance_loss(far, M.MOE_DTYPE_F32, stride, idx.to(DEV), None, T, E, 2, 0, 0.01, 0.1, *o,
                       None, out, M.MOE_DTYPE_F16, stride)
    assert all(torch.equal(a, b) for a, b in zip(o, want))
    assert torch.equal(out.as_strided((T, E), (stride, 1)), want[3].half())


def test_streams_and_graph():
    say("balance: side stream and graphs")
    for T in (40, 700):
        l, idx, mask = (t.to(DEV) for t in draw(T, 96, 4, masked=0.2))
        args = (mask, 4, "sigmoid", 0.01, 0.1)
        want = call(l, idx, *args)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = call(l, idx, *args)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                ws = torch.empty(M.moe_balance_loss_workspace_bytes(T, 96) + 1, dtype=torch.uint8,
                                 device=DEV)
                graphs.append((graph, call(l, idx, *args, ws=ws), ws))
        for i in range(4):
            l.copy_(torch.randn_like(l))
            idx.copy_(torch.randint_like(idx, 0, 96))
            want = call(l, idx, *args)
            graph, outs, _ = graphs[i % 2]
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
