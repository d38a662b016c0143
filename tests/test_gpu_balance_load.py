"""moe_balance_loss where the load and the probabilities lie apart, where no choice
counts, and with gradients scaled beyond fp32."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
from tests import block_util as R
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
U = R.U
SCORES = {"softmax": M.MOE_SCORE_SOFTMAX, "sigmoid": M.MOE_SCORE_SIGMOID}


def call(l, idx, mask, k, score, coef, zcoef=0.0, counts=None, up=None):
    T, E = l.shape
    o = [torch.full((E,), -7, dtype=torch.int32, device=DEV) if counts is None else counts,
         torch.full((E,), -7.0, device=DEV), torch.full((2,), -7.0, device=DEV),
         torch.full((T, E), -7.0, device=DEV)]
    nb = M.moe_balance_loss_workspace_bytes(T, E)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=DEV)
    M.moe_balance_loss(l.to(DEV), M.MOE_DTYPE_F32, E, None if idx is None else idx.to(DEV),
                       None if mask is None else mask.to(DEV), T, E, k, SCORES[score], coef, zcoef,
                       *o[:3], up, o[3], M.MOE_DTYPE_F32, E, ws, nb)
    return [t.cpu() for t in o]


def logits(T, E, seed=0):
    return 1.2 * torch.randn((T, E), generator=torch.Generator().manual_seed(T + 31 * E + seed))


# As in test_gpu_balance: a probability is off by A + 40 half steps where the row's
# logits span A, every sum of values of one sign adds its additions' half steps (24 in a
# row and wave, one a row of a wave, 80 for the joins), and the weights E c / total two.
def room(l):
    return 2 * (96 + 2 * float(l.max() - l.min()) + l.shape[0] / 2048 + 80) * U


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("T,E,k", [(1, 64, 4), (64, 60, 4), (65, 60, 4), (3000, 60, 4), (70, 1000, 2)])
def test_no_choice_counts(T, E, k, score):
    """Every index outside the experts, or given counts of zero: no load, no loss."""
    l = logits(T, E)
    idx = torch.full((T, k), E, dtype=torch.int32)
    idx[:, 0] = -1
    z = R.balance_ref(l, idx, None, E, SCORES[score], 0.5, 0.25)[2][1]
    for args in ((idx, None), (None, torch.zeros(E, dtype=torch.int32, device=DEV))):
        counts, mean, losses, grad = call(l, args[0], None, k, score, 0.5, 0.25, args[1])
        assert (counts == 0).all() and float(losses[0]) == 0.0
        assert abs(float(losses[1]) - z) <= room(l) * z
        assert torch.isfinite(grad).all() and abs(float(mean.double().sum()) - 1.0) < 1e-4
        only = call(l, args[0], None, k, score, 0.5, 0.0, args[1])[3]
        assert (only == 0).all()


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("far", [6.0, 14.0, 30.0])
@pytest.mark.parametrize("T,E", [(20, 64), (700, 64), (700, 512)])
def test_load_on_unlikely_experts(T, E, far, score):
    """All choices on experts whose scores are far below the others': the loss is small,
    a sum of positive terms, and right in itself."""
    l = logits(T, E)
    l[:, 3:5] -= far
    idx = torch.full((T, 2), 3, dtype=torch.int32)
    idx[::3, 1] = 4
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.8).to(torch.uint8)
    mask[0] = 1
    want = R.balance_ref(l, idx, mask, E, SCORES[score], 0.5, 0.0)
    got = call(l, idx, mask, 2, score, 0.5)
    assert torch.equal(got[0].long(), want[0])
    assert abs(float(got[2][0]) - want[2][0]) <= room(l) * want[2][0]
    given = call(l, None, mask, 2, score, 0.5, counts=got[0].to(DEV))
    assert torch.equal(given[2], got[2])


@pytest.mark.parametrize("up", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("T", [5, 130])
def test_masked_stays_zero_whatever_the_scale(T, score, up):
    """A loss scale that overflowed reaches no masked expert and no masked token."""
    E, k = 70, 4
    l = logits(T, E)
    idx = torch.sort(l, dim=1, descending=True)[1][:, :k].int().contiguous()
    l[0, 3], l[0, 69], l[1, :], l[2, 1:] = -np.inf, np.nan, -np.inf, -np.inf
    mask = torch.ones(T, dtype=torch.uint8)
    mask[4] = 0
    grad = call(l, idx, mask, k, score, 0.01, 0.01, up=torch.tensor([up], device=DEV))[3]
    assert grad[0, 3] == 0 and grad[0, 69] == 0 and (grad[1] == 0).all()
    assert (grad[2, 1:] == 0).all() and (grad[4] == 0).all()
    assert not torch.isfinite(grad[3]).any()


@pytest.mark.parametrize("T", [5, 200])
def test_given_counts_are_not_written(T):
    """With tokens, also where all of them are masked."""
    counts = torch.arange(40, dtype=torch.int32, device=DEV)
    got = call(logits(T, 40), None, torch.zeros(T, dtype=torch.uint8), 2, "softmax", 0.1,
               counts=counts.clone())
    assert torch.equal(got[0], counts.cpu()) and all((t == 0).all() for t in got[1:])


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("zcoef", [0.001, 1.0])
def test_largest_logit_with_z_loss(T, score, zcoef):
    """+inf counts as the largest finite value, whose z loss leaves fp32; its gradient
    may too, the other experts' is none of that."""
    E = 40
    l = logits(T, E)
    l[0, 7] = np.inf
    idx = torch.zeros((T, 2), dtype=torch.int32)
    _, _, _, want = R.balance_ref(l, idx, None, E, SCORES[score], 0.0, zcoef)
    counts, mean, losses, grad = call(l, idx, None, 2, score, 0.0, zcoef)
    assert torch.isfinite(mean).all() and losses[0] == 0 and torch.isposinf(losses[1])
    assert (grad[0, :7] == 0).all() and (grad[0, 8:] == 0).all()
    big = float(want[0, 7])
    assert float(grad[0, 7]) == pytest.approx(big, rel=1e-5) if big < 3.4e38 else \
        torch.isposinf(grad[0, 7])
    assert torch.isfinite(grad[1:]).all()
