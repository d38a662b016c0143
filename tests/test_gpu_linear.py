"""moe_linear_f16 and its gradients against the 64-bit definition."""
import pytest
import torch

import int4_weight_only_router_amd as M
from tests import block_util as R
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
U = R.U


def rand(g, *s):
    return torch.randn(s, generator=g, dtype=torch.float32)


def put(x, pad, dtype=torch.float16, fill=7.0):
    wide = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=dtype, device=DEV)
    wide[:, :x.shape[1]] = x.to(DEV, dtype)
    return wide


def f64(t, cols):
    return t.cpu().double()[:, :cols]


def run(x, w, bias, act, residual, m, n, k, dtype, z=None, out=None, pad=0, stream=None):
    dt, code = R.TYPES[dtype]
    if out is None:
        out = torch.full((m, n + pad), -3.0, dtype=dt, device=DEV)
    nb = M.moe_linear_f16_workspace_bytes(m, n, k)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=DEV)
    M.moe_linear_f16(x, x.shape[1], w, w.shape[1], bias, R.ACTS[act], residual,
                     0 if residual is None else residual.shape[1], m, n, k, out, code,
                     out.shape[1], z, 0 if z is None else z.shape[1], ws, nb, stream)
    return out


def sum_bound(k):
    """Worst case of k fp32 additions, in units of the sum of magnitudes."""
    return (k + 16) * U


def check(got, want, bound, l2, what):
    got = got.cpu().double()
    off = (got - want).abs()
    assert (off <= bound).all(), "%s: %.3g of its bound" % (what, float((off / bound).max()))
    norm = float(want.norm())
    if want.numel() >= 1000:   # (few values: no averages)
        assert float(off.norm()) <= l2 * norm, "%s: L2 %.3g" % (what, float(off.norm()) / norm)


def l2_bound(dtype, k, roundings=1):
    """Relative L2 error.  A rounding's error is spread evenly over half a step of a
    value between one and two steps' power: its rms is below half / sqrt(3); fp32 sums
    of k terms of either sign: below sqrt(k) half steps, the partial sums being no
    larger than the result's rms in the mean."""
    h = R.half_step(R.TYPES[dtype][0])
    return (roundings * (h / 3 ** 0.5) ** 2 + k * U * U) ** 0.5


FORWARD = [(1, 64, 64), (1, 5632, 2048), (2, 1, 8), (3, 17, 24), (7, 100, 2000), (8, 33, 2048),
           (15, 257, 72), (16, 1408, 2048), (17, 1408, 2000), (31, 16, 4096), (32, 512, 256),
           (33, 300, 520), (48, 60, 2048), (64, 64, 64), (65, 1000, 8), (100, 2049, 136),
           (128, 5632, 2048), (129, 257, 1032), (200, 5632, 512), (255, 255, 264),
           (333, 1408, 2000), (512, 64, 2048), (777, 60, 2048), (1000, 1000, 1000),
           (1025, 2056, 520), (4096, 64, 2048), (2048, 2048, 128), (4099, 1, 256)]


@pytest.mark.parametrize("dtype,act", [("f16", "silu"), ("f32", "none")])
@pytest.mark.parametrize("m,n,k", FORWARD)
def test_forward(m, n, k, dtype, act):
    say("linear %dx%dx%d %s %s" % (m, n, k, dtype, act))
    g = torch.Generator().manual_seed(m + n + k)
    x, w = put(rand(g, m, k), 8 * (m % 2)), put(0.05 * rand(g, n, k), 8 * (n % 3))
    bias = rand(g, n).to(DEV)
    dt = R.TYPES[dtype][0]
    res = put(rand(g, m, n), n % 2, dt)
    z = torch.full((m, n + 3), -3.0, dtype=torch.float16, device=DEV)
    out = run(x, w, bias, act, res, m, n, k, dtype, z, pad=5)
    torch.cuda.synchronize()
    xv, wv = f64(x, k), f64(w, k)
    zv = xv @ wv.t() + bias.cpu().double()
    size = xv.abs() @ wv.abs().t() + bias.cpu().double().abs()
    want = R.act_ref(zv, act) + f64(res, n)
    e = sum_bound(k) * size
    zb = e + R.half_step(torch.float16) * zv.abs() + R.tiny(torch.float16)
    check(z[:, :n], zv, zb, l2_bound("f16", k), "z")
    # |act'| <= 1.13; the activation itself in fp32: 16 half steps of |z| + 1
    bound = 1.13 * e + 16 * U * (zv.abs() + 1) + 2 * U * f64(res, n).abs() \
        + R.half_step(dt) * (want.abs() + 1.13 * e) + R.tiny(dt)
    # (the residual and the activation change the result's size against the sum's)
    scale = max(1.0, float(size.norm() * 0 + zv.norm()) / max(float(want.norm()), 1e-30))
    check(out[:, :n], want, bound, l2_bound(dtype, k) + scale * 1.13 * l2_bound("f32", k), "out")
    assert (out[:, n:] == -3.0).all() and (z[:, n:] == -3.0).all()
    # without z, in place over the residual: the same bits
    again = run(x, w, bias, act, res, m, n, k, dtype, out=res)
    assert torch.equal(again[:, :n], out[:, :n])


@pytest.mark.parametrize("act", list(R.ACTS))
@pytest.mark.parametrize("m,n,k", [(5, 48, 64), (130, 260, 64)])
def test_activations(act, m, n, k):
    """Over z from -30 to 30, without bias and residual."""
    g = torch.Generator().manual_seed(3)
    x, w = put(rand(g, m, k), 0), put(rand(g, n, k), 0)
    out = run(x, w, None, act, None, m, n, k, "f32")
    zv = f64(x, k) @ f64(w, k).t()
    e = sum_bound(k) * (f64(x, k).abs() @ f64(w, k).abs().t())
    assert float(zv.abs().max()) > 20
    check(out, R.act_ref(zv, act), 1.13 * e + 16 * U * (zv.abs() + 1), 1e-5, act)


@pytest.mark.parametrize("act", list(R.ACTS))
@pytest.mark.parametrize("m", [3, 80])
def test_bad_values(act, m):
    """Infinities and NaN stay in their rows and columns; far values saturate."""
    n, k = 96, 64
    x, w = torch.zeros((m, k)), torch.zeros((n, k))
    x[:, 0], w[:, 0] = 1.0, 1.0
    x[1, 0] = float("nan")
    w[5, 0] = 60000.0
    w[6, 0] = -60000.0
    out = run(put(x, 0), put(w, 0), None, act, None, m, n, k, "f32").cpu()
    rest = [i for i in range(m) if i != 1]
    assert torch.isnan(out[1]).all() and torch.isfinite(out[rest]).all()
    assert (out[rest][:, 5] == 60000.0).all()
    assert (out[rest][:, 6] == (-60000.0 if act == "none" else 0.0)).all()


@pytest.mark.parametrize("m,n,k", [(1, 64, 520), (2, 64, 512), (7, 64, 64), (70, 70, 64)])
def test_subnormal_operands(m, n, k):
    """fp16's subnormals count in full: 2^-20 times 2^10, k times."""
    x = put(torch.full((m, k), 2.0 ** -20), 0)
    w = put(torch.full((n, k), 1024.0), 0)
    out = run(x, w, None, "none", None, m, n, k, "f32")
    assert (out == k * 2.0 ** -10).all()
    out = run(w, x, None, "none", None, n, m, k, "f32")
    assert (out == k * 2.0 ** -10).all()


def test_weights_past_the_end_are_not_read_into_results():
    """NaN all around the operands: rows, columns and padding that a tile covers but
    the product does not hold."""
    for m, n, k in ((5, 40, 72), (70, 70, 72), (300, 300, 136)):
        big = torch.full((m + 300, k + 64), float("nan"), dtype=torch.float16, device=DEV)
        bw = torch.full((n + 300, k + 64), float("nan"), dtype=torch.float16, device=DEV)
        big[:m, :k], bw[:n, :k] = 1.0, 0.5
        out = torch.zeros((m, n), dtype=torch.float32, device=DEV)
        nb = M.moe_linear_f16_workspace_bytes(m, n, k)
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=DEV)
        M.moe_linear_f16(big, k + 64, bw, k + 64, None, 0, None, 0, m, n, k, out,
                         M.MOE_DTYPE_F32, n, None, 0, ws, nb)
        assert (out == 0.5 * k).all()


# ------------------------------------------------------------------ gradients

def backward(dy, z, act, x, w, m, n, k, dtype, dx, dw, db, stream=None, ws=None):
    nb = M.moe_linear_f16_backward_workspace_bytes(m, n, k)
    if ws is None:
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=DEV)
    width = lambda t: 0 if t is None else t.shape[1]  # noqa: E731
    M.moe_linear_f16_backward(dy, dy.shape[1], z, width(z), R.ACTS[act], x, x.shape[1], w,
                              w.shape[1], m, n, k, dx, width(dx), dw, width(dw),
                              R.TYPES[dtype][1], db, ws, nb, stream)
    return ws


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("m,n,k", [(70, 131, 72), (1000, 1003, 264), (2050, 2054, 136),
                                   (4100, 5009, 72), (4100, 8200, 64), (2050, 2055, 2504),
                                   (4100, 5001, 264)])
def test_sums_and_bias_only(m, n, k, bias, dtype):
    """Nothing but the sums and a bias leaves: of every tile's form."""
    say("linear sums %dx%dx%d %s" % (m, n, k, dtype))
    g = torch.Generator().manual_seed(m + n)
    x, w = put(rand(g, m, k), 0), put(0.05 * rand(g, n, k), 8)
    b = rand(g, n).to(DEV) if bias else None
    out = run(x, w, b, "none", None, m, n, k, dtype, pad=n % 4)
    xv, wv = f64(x, k), f64(w, k)
    want, size = xv @ wv.t(), xv.abs() @ wv.abs().t()
    if bias:
        want, size = want + b.cpu().double(), size + b.cpu().double().abs()
    dt = R.TYPES[dtype][0]
    e = sum_bound(k) * size
    check(out[:, :n], want, e + R.half_step(dt) * (want.abs() + e) + R.tiny(dt), l2_bound(dtype, k), "out")
    assert (out[:, n:] == -3.0).all()


BACKWARD = [(1, 64, 64), (2, 1, 8), (3, 17, 24), (16, 1408, 2048), (33, 300, 520), (64, 60, 2048),
            (65, 1000, 8), (130, 257, 1032), (255, 256, 264), (333, 1408, 2000), (777, 60, 2048),
            (1000, 1000, 1000), (1025, 520, 264), (4096, 64, 2048), (4099, 3, 256),
            (33000, 24, 64), (70001, 7, 8), (2050, 2505, 2056), (264, 4100, 5000),
            (4100, 72, 8200)]


@pytest.mark.parametrize("dtype,act", [("f16", "silu"), ("f32", "none"), ("f16", "none")])
@pytest.mark.parametrize("m,n,k", BACKWARD)
def test_backward(m, n, k, dtype, act):
    say("linear backward %dx%dx%d %s %s" % (m, n, k, dtype, act))
    g = torch.Generator().manual_seed(m + n + k)
    dt = R.TYPES[dtype][0]
    x, w = put(rand(g, m, k), 8 * (m % 2)), put(0.05 * rand(g, n, k), 8 * (n % 3))
    dy, z = put(rand(g, m, n), n % 5), put(2.0 * rand(g, m, n), n % 3)
    dx, dw = (torch.full((r, k + 5), -3.0, dtype=dt, device=DEV) for r in (m, n))
    db = torch.full((n,), -3.0, device=DEV)
    backward(dy, z if act != "none" else None, act, x, w, m, n, k, dtype, dx, dw, db)
    torch.cuda.synchronize()
    slope = R.act_grad_ref(f64(z, n), act)
    dz = f64(dy, n) * slope
    # of dz: fp32 activation (16 half steps of |dy|), one rounding to fp16
    soft = act != "none"
    ez = (16 * U * f64(dy, n).abs() + R.half_step(torch.float16) * dz.abs()
          + R.tiny(torch.float16)) if soft else torch.zeros_like(dz)
    h, t = R.half_step(dt), R.tiny(dt)
    roundings = 2 if soft else 1
    for got, want, size, es, terms in (
            (dx, dz @ f64(w, k), dz.abs() @ f64(w, k).abs(), ez @ f64(w, k).abs(), n),
            (dw, dz.t() @ f64(x, k), dz.abs().t() @ f64(x, k).abs(), ez.t() @ f64(x, k).abs(), m)):
        e = sum_bound(terms) * (size + es) + es
        l2 = l2_bound(dtype, terms, roundings) + 4 * U
        check(got[:, :k], want, e + h * (want.abs() + e) + t, l2, "dx" if terms == n else "dw")
        assert (got[:, k:] == -3.0).all()
    e = sum_bound(m) * dz.abs().sum(0) + 16 * U * f64(dy, n).abs().sum(0)
    check(db, dz.sum(0), e + U * dz.sum(0).abs(), 1.0, "dbias")
    # each alone: the same bits
    for i in range(3):
        alone = [torch.full_like(b, -3.0) if i == j else None for j, b in enumerate((dx, dw, db))]
        backward(dy, z if soft else None, act, x, w, m, n, k, dtype, *alone)
        assert torch.equal(alone[i], (dx, dw, db)[i])


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("m,n,k", [(1, 5632, 2048), (3, 17, 24), (4, 1407, 520), (100, 63, 520),
                                   (127, 64, 1000), (4099, 16, 32), (20, 1000, 64)])
def test_backward_few_values(m, n, k, act):
    """No rounding but the gradients' own where few values are: dz carries its rest."""
    say("linear backward, few values: %dx%dx%d %s" % (m, n, k, act))
    g = torch.Generator().manual_seed(m + n)
    x, w = put(rand(g, m, k), 0), put(0.05 * rand(g, n, k), 8)
    dy, z = put(rand(g, m, n), 1), put(2 * rand(g, m, n), 3)
    dx, dw = (torch.full((r, k + 5), -3.0, dtype=torch.float16, device=DEV) for r in (m, n))
    backward(dy, z, act, x, w, m, n, k, "f16", dx, dw, None)
    torch.cuda.synchronize()
    zv = f64(z, n)
    dz = f64(dy, n) * R.act_grad_ref(zv, act)
    # dz in fp32 (16 half steps of dy as elsewhere) and the rest's own rounding: the first
    # fp16 lies up to a whole step before dz, the rest is up to 2^-10 of it and rounded
    # by 2^-11 of itself, or to the smallest subnormal
    ez = 16 * U * f64(dy, n).abs() + 2.0 ** -21 * dz.abs() + R.tiny(torch.float16)
    h, t = R.half_step(torch.float16), R.tiny(torch.float16)
    for got, want, size, es, terms in (
            (dx, dz @ f64(w, k), dz.abs() @ f64(w, k).abs(), ez @ f64(w, k).abs(), 2 * n),
            (dw, dz.t() @ f64(x, k), dz.abs().t() @ f64(x, k).abs(), ez.t() @ f64(x, k).abs(), 2 * m)):
        e = sum_bound(terms) * (size + es) + es
        check(got[:, :k], want, e + h * (want.abs() + e) + t, l2_bound("f16", terms) + 8 * U,
              "dx" if terms == 2 * n else "dw")
        assert (got[:, k:] == -3.0).all()


def test_backward_few_values_not_finite():
    """An infinite weight and a gradient beyond fp16 stay infinities, with their signs."""
    n, k = 70, 64
    g = torch.Generator().manual_seed(3)
    x, w = put(rand(g, 2, k), 0), put(rand(g, n, k), 0)
    dy, z = put(rand(g, 2, n).abs() + 0.5, 0), put(rand(g, 2, n).abs() + 4, 0)   # act' about one
    w[n - 1, 5], w[3, 9] = float("inf"), -float("inf")
    dy[1, 7] = float("inf")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    backward(dy, z, "silu", x, w, 2, n, k, "f16", dx, dw, None)
    assert dx[0, 5] == float("inf") and dx[0, 9] == -float("inf")
    cols = [i for i in range(k) if i not in (5, 9)]
    assert torch.isfinite(dx[0, cols]).all()
    assert torch.equal(dx[1, cols], torch.sign(w[7, cols].float()).half() * float("inf"))
    assert torch.isinf(dw[7]).all() and torch.isfinite(dw[:7]).all() and torch.isfinite(dw[8:]).all()



@pytest.mark.parametrize("act", list(R.ACTS))
def test_activation_gradients(act):
    """dz through the unit matrix: every act' over z from -20 to 20, against the
    definition's derivative and against differences."""
    n, m = 64, 200
    z = torch.linspace(-20.0, 20.0, m * n).reshape(m, n)
    z[0, 0], z[0, 1] = 0.0, -0.0
    zd, dy = put(z, 0), put(torch.ones((m, n)), 0)
    eye = put(torch.eye(n), 0)
    dx = torch.empty((m, n), dtype=torch.float16, device=DEV)
    db = torch.empty(n, device=DEV)
    x = put(torch.zeros((m, n)), 0)
    backward(dy, zd if act != "none" else None, act, x, eye, m, n, n, "f16", dx, None, db)
    zv = f64(zd, n)
    want = R.act_grad_ref(zv, act)
    bound = 16 * U + R.half_step(torch.float16) * want.abs() + R.tiny(torch.float16)
    assert ((dx.cpu().double() - want).abs() <= 2 * bound).all()
    if act != "relu":
        h = 1e-5   # third derivatives are below 3: the difference is off by h^2 / 2
        diff = (R.act_ref(zv + h, act) - R.act_ref(zv - h, act)) / (2 * h)
        assert ((dx.cpu().double() - diff).abs() <= 2 * bound + h * h + 1e-9).all()


def test_backward_no_rows():
    dw, db = torch.full((5, 16), 3.0, dtype=torch.float16, device=DEV), torch.ones(5, device=DEV)
    M.moe_linear_f16_backward(None, 5, None, 0, M.MOE_ACT_NONE, None, 16, None, 16, 0, 5, 16, None,
                              0, dw, 16, M.MOE_DTYPE_F16, db)
    assert (dw == 0).all() and (db == 0).all()


def test_streams_and_graph():
    say("linear: side stream and graphs")
    for m, n, k in ((4, 320, 512), (300, 60, 1024)):
        g = torch.Generator().manual_seed(9)
        x, w, dy = put(rand(g, m, k), 0), put(0.05 * rand(g, n, k), 0), put(rand(g, m, n), 0)

        def passes(stream=None, ws=(None, None)):
            z = torch.empty((m, n), dtype=torch.float16, device=DEV)
            out = run(x, w, None, "gelu", None, m, n, k, "f16", z, stream=stream)
            o = [torch.empty_like(x), torch.empty_like(w), torch.empty(n, device=DEV)]
            keep = backward(dy, z, "gelu", x, w, m, n, k, "f16", *o, stream=stream)
            return [z, out] + o, keep
        want, _ = passes()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got, _ = passes()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                kept = passes()
            graphs.append((graph, kept))
        for i in range(4):
            x.copy_(torch.randn_like(x))
            dy.copy_(torch.randn_like(dy))
            want, _ = passes()
            graph, (outs, _) = graphs[i % 2]
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
