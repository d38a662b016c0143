"""What the L2 bound of the FP8 experts accepts and rejects, on the CPU: the
operator in fp32 as it is, and wrong forms of it, at the sizes of real layers."""
import numpy as np
import pytest

from tests import fp8_strict as S
from tests import fp8_util as R

F = np.float32


def _weights(r, n, c):
    return R.quantize(r.normal(0, 0.02, (n, c)).astype(F), 128, False)


def _product(xq, xs, wq, ws, cast=lambda a: a):
    """fp32 sums block by block."""
    n, K = xq.shape
    acc = np.zeros((n, wq.shape[0]), F)
    for b in range(R.blocks(K)):
        c = slice(128 * b, min(K, 128 * b + 128))
        s = xs[:, b, None] * np.repeat(ws[:, b], 128)[None, :wq.shape[0]]
        acc = cast(acc + (xq[:, c].astype(F) @ wq[:, c].astype(F).T) * s)
    return acc


def _bf16(a):
    b = a.view(np.uint32)
    return ((b + 0x7fff + ((b >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(F)


def _experts(x, wg, wu, wd, wrong=None):
    cast = _bf16 if wrong == "bf16 sums" else lambda a: a
    xq, xs = R.quantize(x, 1, wrong != "scales not powers of two")
    g = _product(xq, xs, *wg, cast)
    u = _product(xq, xs, *wu, cast)
    if wrong == "gate off by 1%":
        g = g * F(1.01)
    if wrong == "gate and up swapped":
        g, u = u, g
    h = g / (F(1) + np.exp(-g)) * u
    if wrong == "column of h lost":
        h[:, np.abs(h[0]).argmax()] = 0
    if wrong == "h in bf16":
        h = _bf16(h)
    hq, hs = R.quantize(h, 1, True)
    if wrong == "h not quantised":
        hq, hs = h, np.ones_like(hs)
    if wrong == "block of h lost":
        hq[:, -128:] = 0
    if wrong == "codes cut":
        below = np.abs(hq) > np.abs(h / R.spread(hs, 1, *h.shape))
        hq = np.where(below, np.sign(hq) * (np.abs(hq) - R.e4m3_step(hq)), hq)
    y = _product(hq, hs, *wd, cast)
    if wrong == "y off by 2%":
        y = y * F(1.02)
    return y.astype(np.float16).astype(np.float64)


SIZES = [(1, 2048, 1024), (11, 2048, 1408), (70, 2048, 512), (3, 256, 192)]
WRONG = ["h not quantised", "gate off by 1%", "y off by 2%", "bf16 sums", "column of h lost",
         "gate and up swapped", "scales not powers of two", "block of h lost", "codes cut"]


@pytest.fixture(scope="module")
def cases():
    made = {}

    def get(n, H, I):
        if (n, H, I) not in made:
            r = np.random.default_rng(n + H + I)
            w = (_weights(r, I, H), _weights(r, I, H), _weights(r, H, I))
            x = r.normal(0, 1, (n, H)).astype(np.float16).astype(F)
            made[n, H, I] = x, w, S.experts_l2(x, *w, False), S.experts_l2(x, *w, True)
        return made[n, H, I]
    return get


@pytest.mark.parametrize("n,H,I", SIZES)
def test_right_form_fits(cases, n, H, I):
    x, w, fp32, runs = cases(n, H, I)
    err = np.linalg.norm(_experts(x, *w) - fp32[0], axis=1)
    assert np.all(err <= fp32[1]) and np.all(fp32[1] <= runs[1])
    # no blanket (a row whose block scale may be either has more room than most)
    assert np.median(runs[1] / np.linalg.norm(fp32[0], axis=1)) <= 0.02


@pytest.mark.parametrize("wrong", WRONG)
@pytest.mark.parametrize("n,H,I", SIZES)
def test_wrong_forms_do_not(cases, n, H, I, wrong):
    x, w, fp32, runs = cases(n, H, I)
    y = _experts(x, *w, wrong)
    for ref, allowed in (fp32, runs):
        assert np.any(np.linalg.norm(y - ref, axis=1) > allowed)
