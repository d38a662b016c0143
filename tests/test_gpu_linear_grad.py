"""Gradients of moe_linear_f16 whose dz the caller has not asked to be rounded: as
accurate as their own rounding at every size, for small values too, and what z and
weights that are not finite make of them."""
import pytest
import torch

import int4_weight_only_router_amd as M
from tests import block_util as R
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = R.U
F16 = torch.float16
SOFT = ["silu", "gelu", "gelu_tanh"]


def rand(g, *s):
    return torch.randn(s, generator=g, dtype=torch.float32)


def put(x, pad=0):
    wide = torch.full((x.shape[0], x.shape[1] + pad), 7.0, dtype=F16, device=DEV)
    wide[:, :x.shape[1]] = x.to(DEV, F16)
    return wide


def backward(dy, z, act, x, w, m, n, k, out, dtype=M.MOE_DTYPE_F16, fill=0):
    """out: dx, dw, dbias (or None each); `fill`: the workspace's bytes before the call."""
    nb = M.moe_linear_f16_backward_workspace_bytes(m, n, k)
    ws = torch.full((max(nb, 1),), fill, dtype=torch.uint8, device=DEV)
    ld = [0 if t is None else t.shape[1] for t in (dy, z, x, w) + tuple(out[:2])]
    M.moe_linear_f16_backward(dy, ld[0], z, ld[1], R.ACTS[act], x, ld[2], w, ld[3], m, n, k,
                              out[0], ld[4], out[1], ld[5], dtype, out[2], ws, nb)
    return out


def inputs(m, n, k, scale=1.0):
    g = torch.Generator().manual_seed(m + n + k)
    return (put(scale * rand(g, m, n), n % 5), put(2.0 * rand(g, m, n), n % 3),
            put(rand(g, m, k), 8 * (m % 2)), put(0.05 * rand(g, n, k), 8 * (n % 3)))


def outputs(m, n, k):
    return [torch.full((r, k + 3), -3.0, dtype=F16, device=DEV) for r in (m, n)] + \
        [torch.full((n,), -3.0, device=DEV)]


def wide(t, cols):
    return t[:, :cols].double()


def definition(dy, z, act, x, w, m, n, k):
    """dz, dx and dw in 64 bits."""
    dz = wide(dy, n) * R.act_grad_ref(wide(z, n), act)
    return dz, dz @ wide(w, k), dz.t() @ wide(x, k)


def ratio(got, want):
    """The error's L2 norm against that of rounding the exact values."""
    own = (want.to(F16).double() - want).norm()
    return float((got.double() - want).norm() / own)


# The products of every form of a tile, whole and in parts of k, with odd and even
# columns, up to those of a prompt.
SIZES = [(17, 5632, 2048), (64, 2048, 5632), (333, 1408, 2000), (333, 1407, 2000), (700, 60, 2048),
         (1000, 1003, 1000), (1025, 520, 264), (2050, 2505, 2056), (264, 4100, 5000),
         (4100, 72, 8200), (2048, 2048, 2048), (4096, 5632, 2048), (2270, 250, 4600), (2000, 40, 264)]


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_no_rounding_but_the_results(m, n, k, act):
    """dz in one fp16 adds as much again (a ratio of 1.4).  As the sum of two it is off
    by 2^-21 of itself, and the fp32 sums by sqrt(terms) half steps: together below 2%
    of a rounding's rms, 2^-11 / sqrt(6) at least; over 2^14 values a rounding's own
    norm varies by 0.4%."""
    say("gradients %dx%dx%d %s" % (m, n, k, act))
    dy, z, x, w = inputs(m, n, k)
    dx, dw, db = backward(dy, z, act, x, w, m, n, k, outputs(m, n, k))
    dz, want_x, want_w = definition(dy, z, act, x, w, m, n, k)
    assert ratio(dx[:, :k], want_x) < 1.03, "dx %.3f" % ratio(dx[:, :k], want_x)
    assert ratio(dw[:, :k], want_w) < 1.03, "dw %.3f" % ratio(dw[:, :k], want_w)
    assert (dx[:, k:] == -3.0).all() and (dw[:, k:] == -3.0).all()
    # 64 rows or M / 512 of them a part, then 16 parts at a time and their sums: fewer
    # than 200 additions in sequence of values of either sign, each off by half a step
    # of a partial sum no larger than the whole in the mean; dz itself by 16 of |dy|
    size = dz.pow(2).sum(0).sqrt() + dz.sum(0).abs()
    room = 16 * U * (200 ** 0.5 * size + wide(dy, n).pow(2).sum(0).sqrt() * 4)
    assert ((db.double() - dz.sum(0)).norm() <= room.norm())
    assert float(db.double().norm()) > 0
    # again, over a workspace that held something else: the same bits
    again = backward(dy, z, act, x, w, m, n, k, outputs(m, n, k), fill=0xFF)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("act", SOFT)
@pytest.mark.parametrize("m,n,k", [(3, 17, 24), (300, 1003, 264), (2050, 2505, 2056)])
def test_within_the_bound(m, n, k, act):
    """Value by value: dz in fp32 (16 half steps of dy), its rest's rounding, fp32 sums of
    2 terms a k, one rounding."""
    dy, z, x, w = inputs(m, n, k)
    dx, dw, _ = backward(dy, z, act, x, w, m, n, k, outputs(m, n, k))
    dz, want_x, want_w = definition(dy, z, act, x, w, m, n, k)
    ez = 16 * U * wide(dy, n).abs() + 2.0 ** -21 * dz.abs() + R.tiny(F16)
    h = R.half_step(F16)
    for got, want, size, es, terms in (
            (dx, want_x, dz.abs() @ wide(w, k).abs(), ez @ wide(w, k).abs(), 2 * n),
            (dw, want_w, dz.abs().t() @ wide(x, k).abs(), ez.t() @ wide(x, k).abs(), 2 * m)):
        e = (terms + 16) * U * (size + es) + es
        off = (got[:, :k].double() - want).abs()
        assert (off <= e + h * (want.abs() + e) + R.tiny(F16)).all()


@pytest.mark.parametrize("act", SOFT)
@pytest.mark.parametrize("scale", [2.0 ** -10, 2.0 ** -13, 1e-5, 2.0 ** -22])
@pytest.mark.parametrize("m", [3, 200])
def test_small_gradients(m, scale, act):
    """dz below fp16's normal values, through the unit matrix: the sum of the two fp16 is
    the multiple of 2^-24 next to it, off by 2^-25 (and dz in fp32 by 16 half steps of
    dy), and dx rounds that once more where it is 2^-13 or above."""
    n = 256
    dy, z, x, _ = inputs(m, n, n, scale)
    z[:, :n] = (z[:, :n].float().abs() + 4).half()   # act' about one
    eye = put(torch.eye(n))
    dx, dw, _ = backward(dy, z, act, x, eye, m, n, n, outputs(m, n, n))
    dz, want, want_w = definition(dy, z, act, x, eye, m, n, n)
    bound = 2.0 ** -25 + 17 * U * wide(dy, n).abs() + R.half_step(F16) * want.abs()
    small = want.abs() < 2.0 ** -13
    bound[small] -= R.half_step(F16) * want.abs()[small]
    assert ((dx[:, :n].double() - want).abs() <= bound).all()
    es = (2.0 ** -25 + 17 * U * wide(dy, n).abs()).t() @ wide(x, n).abs()
    e = es + (2 * m + 16) * U * (dz.abs().t() @ wide(x, n).abs() + es)
    assert ((dw[:, :n].double() - want_w).abs()
            <= e + R.half_step(F16) * (want_w.abs() + e) + R.tiny(F16)).all()


@pytest.mark.parametrize("act", SOFT)
def test_steps_of_the_smallest_values(act):
    """Every multiple of 2^-24 up to 2^-13 comes through as it is."""
    m, n = 32, 64
    steps = torch.arange(1, m * n + 1).reshape(m, n).double() * 2.0 ** -24
    steps[::2] *= -1
    dy, z = put(steps.float()), put(torch.full((m, n), 60.0))   # act' is one
    eye, x = put(torch.eye(n)), put(torch.zeros((m, n)))
    dx, _, _ = backward(dy, z, act, x, eye, m, n, n, outputs(m, n, n))
    assert torch.equal(dx[:, :n].double().cpu(), steps)


@pytest.mark.parametrize("m,n,k", [(2, 70, 64), (300, 1000, 264), (300, 1001, 264), (4096, 512, 2048)])
def test_infinite_weights(m, n, k):
    """An infinite weight and a gradient beyond fp16 stay infinities, with their signs."""
    g = torch.Generator().manual_seed(m)
    x, w = rand(g, m, k), 0.05 * rand(g, n, k)
    dy, z = rand(g, m, n).abs() + 0.5, rand(g, m, n).abs() + 4   # act' about one
    w[n - 1, 5], w[3, 9] = float("inf"), -float("inf")
    dy[1, 7] = float("inf")
    x, w, dy, z = put(x), put(w), put(dy), put(z)
    dx, dw, _ = backward(dy, z, "silu", x, w, m, n, k, outputs(m, n, k))
    rows = [i for i in range(m) if i != 1]
    assert (dx[rows][:, 5] == float("inf")).all() and (dx[rows][:, 9] == -float("inf")).all()
    cols = [i for i in range(k) if i not in (5, 9)]
    assert torch.isfinite(dx[rows][:, cols]).all()
    assert torch.equal(dx[1, cols], torch.sign(w[7, cols].float()).half() * float("inf"))
    assert torch.isinf(dw[7, :k]).all()
    assert torch.isfinite(dw[:7]).all() and torch.isfinite(dw[8:]).all()


@pytest.mark.parametrize("act", SOFT + ["relu"])
@pytest.mark.parametrize("m", [4, 200])
def test_z_beyond_fp16(act, m):
    """A z that left fp16's range arrives as an infinity; the derivative there is its
    limit, one or zero, and spoils no other value of the row.  NaN stays NaN."""
    n = 64
    dy, z = torch.full((m, n), 0.5), torch.full((m, n), 30.0)
    z[1, 3], z[1, 4], z[2, 7] = float("inf"), -float("inf"), float("nan")
    z[3, 0], z[3, 1] = 65504.0, -65504.0
    want = torch.full((m, n), 0.5)
    want[1, 4], want[3, 1] = 0.0, 0.0
    eye, x = put(torch.eye(n)), put(torch.zeros((m, n)))
    dx, _, db = backward(put(dy), put(z), act, x, eye, m, n, n, outputs(m, n, n))
    keep = [i for i in range(m) if i != 2]
    assert torch.equal(dx[keep][:, :n].cpu().float(), want[keep])
    if act != "relu":
        assert torch.isnan(dx[2, :n]).all()   # (NaN times the unit matrix's zeros)
        assert torch.isnan(db[7]) and torch.isfinite(db[[i for i in range(n) if i != 7]]).all()


@pytest.mark.parametrize("act", list(R.ACTS))
@pytest.mark.parametrize("m,n,k", [(3, 17, 24), (333, 1408, 2000), (2050, 2505, 2056)])
def test_rounded_dz(m, n, k, act):
    """MOE_DZ_F16: dz in one fp16.  Value by value within that rounding, and where dz is
    fp16 as it is (no activation, ReLU) the same bits as without the flag."""
    dy, z, x, w = inputs(m, n, k)
    if act == "none":
        z = None
    a = backward(dy, z, act, x, w, m, n, k, outputs(m, n, k), M.MOE_DTYPE_F16 | M.MOE_DZ_F16)
    b = backward(dy, z, act, x, w, m, n, k, outputs(m, n, k))
    assert torch.equal(a[2], b[2])
    if act in ("none", "relu"):
        assert all(torch.equal(s, t) for s, t in zip(a, b))
        return
    dz, want_x, want_w = definition(dy, z, act, x, w, m, n, k)
    h = R.half_step(F16)
    ez = 16 * U * wide(dy, n).abs() + h * dz.abs() + R.tiny(F16)
    for got, want, size, es, terms in (
            (a[0], want_x, dz.abs() @ wide(w, k).abs(), ez @ wide(w, k).abs(), n),
            (a[1], want_w, dz.abs().t() @ wide(x, k).abs(), ez.t() @ wide(x, k).abs(), m)):
        e = (terms + 16) * U * (size + es) + es
        off = (got[:, :k].double() - want).abs()
        assert (off <= e + h * (want.abs() + e) + R.tiny(F16)).all()
