"""moe_block_norm and its gradients against the 64-bit definition."""
import itertools

import pytest
import torch

import int4_weight_only_router_amd as M
from tests import block_util as R
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

NAMES = ("y", "residual", "gate", "post_w", "post_b", "pre_w", "pre_b")


def case(**kw):
    c = dict(T=5, H=512, kind="rms", post=True, gate="column", bias=True, offset=False,
             scale=0.75, eps=1e-5, dtype="f16", w_dtype="f16", pad=0, residual=True)
    c.update(kw)
    if "w_dtype" not in kw:
        c["w_dtype"] = c["dtype"]
    return c


def name(c):
    return "-".join(str(v) for v in c.values())


def rows(x, pad, dtype, fill=7.0):
    """x as rows of a wider buffer whose other columns hold `fill`."""
    wide = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=dtype, device=DEV)
    wide[:, :x.shape[1]] = x.to(dtype)
    return wide


def inputs(c, seed=0):
    """Device tensors (rows with their padding) and their values in 64 bits."""
    g = torch.Generator().manual_seed(1000 * c["T"] + c["H"] + seed)
    T, H, dt, wt = c["T"], c["H"], R.TYPES[c["dtype"]][0], R.TYPES[c["w_dtype"]][0]
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    d = {n: None for n in NAMES}
    d["y"] = rows(1.5 * r(T, H) + 0.25, c["pad"], dt)
    if c["residual"]:
        d["residual"] = rows(2.0 * r(T, H) - 0.5, c["pad"], dt)
    if c["gate"] == "column":
        d["gate"] = r(1, H).to(DEV, dt)
    elif c["gate"] == "token":
        d["gate"] = rows(r(T, H), c["pad"], dt)
    weight = lambda: (r(H) * 0.2 + (0.0 if c["offset"] else 1.0)).to(DEV, wt)  # noqa: E731
    d["pre_w"] = weight()
    d["post_w"] = weight() if c["post"] else None
    if c["bias"]:
        d["pre_b"] = r(H).to(DEV, wt)
        d["post_b"] = r(H).to(DEV, wt) if c["post"] else None
    v = {n: None if t is None else t.cpu().double()[..., :H] for n, t in d.items()}
    return d, v


def ld(t):
    return 0 if t is None else t.shape[-1]


def common(c):
    """dtype, w_dtype, kind, flags, eps, T, H."""
    flags = (M.MOE_NORM_POST if c["post"] else 0) | (M.MOE_NORM_UNIT_OFFSET if c["offset"] else 0)
    return (R.TYPES[c["dtype"]][1], R.TYPES[c["w_dtype"]][1],
            M.MOE_NORM_RMS if c["kind"] == "rms" else M.MOE_NORM_LAYER, flags, c["eps"], c["T"],
            c["H"])


def ldg(c, d):
    return ld(d["gate"]) if c["gate"] == "token" else 0


def forward(c, d, out, n, stream=None):
    M.moe_block_norm(d["y"], ld(d["y"]), d["residual"], ld(d["residual"]), d["gate"], ldg(c, d),
                     c["scale"], d["post_w"], d["post_b"], d["pre_w"] if n is not None else None,
                     d["pre_b"] if n is not None else None, *common(c), out, ld(out), n, ld(n),
                     stream)


# 48 roundings at most lie between an input and an output (the sums' partial sums
# of 32 columns and the wave's steps among them), each half a step of a value no
# larger than the sizes of block_util; 64 leaves room for the root and the quotients
FORWARD_STEPS = 64


def check(got, want, size, steps, dtype, what):
    got = got.cpu().double()
    bound = R.half_step(dtype) * want.abs() + steps * R.U * (1 + R.half_step(dtype)) * size \
        + R.tiny(dtype)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        what, int(bad.sum()), bad.numel(), float(((got - want).abs() / bound).max()))


FORWARD = [case(T=T, H=H) for T, H in ((1, 2048), (2, 1), (3, 7), (5, 8), (4, 63), (6, 511),
                                       (3, 513), (33, 1000), (9, 1024), (7, 1025), (1027, 2048),
                                       (3, 2049), (5, 4096), (2, 4097), (3, 8192), (2, 8191))]
FORWARD += [case(T=7, H=H, kind=k, dtype=d, gate=g, post=p, bias=b, offset=o, pad=pad)
            for (H, pad), (k, d), (g, p, b, o) in itertools.product(
                ((264, 0), (777, 5), (2304, 8)),
                (("rms", "bf16"), ("layer", "f32"), ("layer", "f16")),
                (("none", False, False, False), ("token", True, True, True),
                 ("column", False, True, True), ("token", False, False, False)))]
FORWARD += [case(dtype="f16", w_dtype="f32", H=1032), case(dtype="bf16", w_dtype="f32", H=2050),
            case(eps=0.0), case(scale=0.0), case(scale=-2.0, gate="none"), case(residual=False),
            case(kind="layer", eps=1.0, H=1)]


@pytest.mark.parametrize("c", FORWARD, ids=name)
def test_forward(c):
    d, v = inputs(c)
    dt, H = R.TYPES[c["dtype"]][0], c["H"]
    out, n = (torch.full((c["T"], H + c["pad"]), -3.0, dtype=dt, device=DEV) for _ in range(2))
    forward(c, d, out, n)
    torch.cuda.synchronize()
    r, m = R.block_norm_ref(c, v)
    sr, sm = R.block_norm_sizes(c, v)
    check(out[:, :H], r, sr, FORWARD_STEPS, dt, "r")
    check(n[:, :H], m, sm, FORWARD_STEPS, dt, "n")
    assert (out[:, H:] == -3.0).all() and (n[:, H:] == -3.0).all()   # the rows' padding
    # one output at a time: the same bits
    o2, n2 = torch.full_like(out, -3.0), torch.full_like(n, -3.0)
    forward(c, d, o2, None)
    forward(c, d, None, n2)
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(n2, n)


def test_norm_without_block():
    """y absent: only the pre-norm of the residual; weights absent: ones and zeros."""
    c = case(post=False, gate="none", bias=False, H=1000, T=9)
    d, v = inputs(c)
    d["y"] = v["y"] = d["pre_w"] = v["pre_w"] = None
    n = torch.empty((9, 1000), dtype=torch.float16, device=DEV)
    forward(c, d, None, n)
    r, m = R.block_norm_ref(c, v)
    check(n, m, R.block_norm_sizes(c, v)[1], FORWARD_STEPS, torch.float16, "n")
    # the offset does not apply to a weight that is not there
    n2 = torch.empty_like(n)
    forward(dict(c, offset=True), d, None, n2)
    assert torch.equal(n, n2)


@pytest.mark.parametrize("H", [512, 2048, 4096, 777])
def test_in_place(H):
    c = case(H=H, T=11, gate="token")
    d, _ = inputs(c)
    out, n = torch.empty_like(d["y"]), torch.empty_like(d["y"])
    forward(c, d, out, n)
    e = {k: None if t is None else t.clone() for k, t in d.items()}
    forward(c, e, e["residual"], e["y"])
    assert torch.equal(e["residual"], out) and torch.equal(e["y"], n)


@pytest.mark.parametrize("H", [512, 4096])
def test_bad_rows_stay_alone(H):
    c = case(H=H, T=8)
    d, _ = inputs(c)
    out, n = torch.empty_like(d["y"]), torch.empty_like(d["y"])
    forward(c, d, out, n)
    d["y"][2, 3], d["residual"][5, H - 1] = float("nan"), float("inf")
    o2, n2 = torch.empty_like(out), torch.empty_like(n)
    forward(c, d, o2, n2)
    good = [0, 1, 3, 4, 6, 7]
    assert torch.equal(o2[good], out[good]) and torch.equal(n2[good], n[good])
    assert not torch.isfinite(n2[[2, 5]]).all(dim=1).any()


def test_far_rows():
    """Rows whose offsets pass 2^32 bytes and 2^31 elements."""
    H, stride = 512, 3 << 29
    wide = torch.empty(2 * stride + H, dtype=torch.float16, device=DEV)
    res = wide.as_strided((3, H), (stride, 1))
    res.copy_(torch.randn((3, H), generator=torch.Generator().manual_seed(4)))
    n, near = (torch.empty((3, H), dtype=torch.float16, device=DEV) for _ in range(2))
    args = (None, 0, 1.0, None, None, None, None, M.MOE_DTYPE_F16, M.MOE_DTYPE_F16,
            M.MOE_NORM_RMS, 0, 1e-5, 3, H)
    M.moe_block_norm(None, 0, res, stride, *args, None, 0, n, H)
    M.moe_block_norm(None, 0, res.contiguous(), H, *args, None, 0, near, H)
    assert torch.equal(n, near) and torch.isfinite(n).all()


# ------------------------------------------------------------------ gradients

def backward(c, d, dout, dn, out, stream=None, ws=None):
    """out: dy, dresidual, dgate, dpost_w, dpost_b, dpre_w, dpre_b."""
    nb = M.moe_block_norm_backward_workspace_bytes(c["T"], c["H"])
    if ws is None:
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=DEV)
    M.moe_block_norm_backward(dout, ld(dout), dn, ld(dn), d["y"], ld(d["y"]), d["residual"],
                              ld(d["residual"]), d["gate"], ldg(c, d), c["scale"], d["post_w"],
                              d["post_b"], d["pre_w"] if dn is not None else None, *common(c),
                              *out, ws, nb, stream)
    return ws


def gradient_buffers(c, d, dn=True):
    like = lambda t: None if t is None else torch.full_like(t, -3.0)  # noqa: E731
    sums = lambda t: None if t is None else torch.full((c["H"],), -3.0, device=DEV)  # noqa: E731
    dgate = like(d["gate"]) if c["gate"] == "token" else sums(d["gate"])
    return [like(d["y"]), like(d["residual"]), dgate, sums(d["post_w"]), sums(d["post_b"]),
            sums(d["pre_w"]) if dn else None, sums(d["pre_b"]) if dn else None]


def reference(c, v, dout, dn):
    leaf = {k: None if t is None else t.clone().requires_grad_(True) for k, t in v.items()}
    r, n = R.block_norm_ref(c, leaf)
    loss = 0.0
    if dout is not None:
        loss = loss + (r * dout).sum()
    if dn is not None:
        loss = loss + (n * dn).sum()
    names = [k for k in NAMES if leaf[k] is not None and (dn is not None or k[:3] != "pre")]
    return dict(zip(names, torch.autograd.grad(loss, [leaf[k] for k in names])))


def sizes(c, v, dout, dn):
    """Sizes of the gradients: the backward formulas with every term in magnitude."""
    H, layer = c["H"], c["kind"] == "layer"
    one = 1.0 if c["offset"] else 0.0

    def stats(x, size):
        if layer:
            size = size + size.mean(-1, keepdim=True)
            x = x - x.mean(-1, keepdim=True)
        rho = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + c["eps"])
        m = x * rho
        dm = rho * size + m.abs() * (1.0 + rho * (m.abs() * size).mean(-1, keepdim=True))
        return m.abs() + dm, rho * (1.0 + rho * (m.abs() * size).mean(-1, keepdim=True))

    def through(g, m, rho):
        return rho * (g + m * (g * m).mean(-1, keepdim=True)
                      + (g.mean(-1, keepdim=True) if layer else 0.0))

    sr, _ = R.block_norm_sizes(c, v)
    r = R.block_norm_ref(c, v)[0]
    dr, out = torch.zeros_like(sr), {}
    if dout is not None:
        dr = dr + dout.abs()
    if dn is not None:
        m, rho = stats(r, sr)
        out["pre_w"], out["pre_b"] = (dn.abs() * m).sum(0), dn.abs().sum(0)
        w = 1.0 if v["pre_w"] is None else (v["pre_w"] + one).abs()
        dr = dr + through(dn.abs() * w, m, rho)
    out["residual"] = dr
    if v["y"] is None:
        return out
    du = abs(c["scale"]) * dr
    m, rho = stats(v["y"], v["y"].abs()) if c["post"] else (v["y"].abs(), None)
    w = 1.0 if v["post_w"] is None else (v["post_w"] + one).abs()
    u = m * w + (0.0 if v["post_b"] is None else v["post_b"].abs()) if c["post"] else m
    out["gate"] = du * u if c["gate"] == "token" else (du * u).sum(0, keepdim=True)
    if v["gate"] is not None:
        du = du * v["gate"].abs()
    if c["post"]:
        out["post_w"], out["post_b"] = (du * m).sum(0), du.sum(0)
        du = through(du * w, m, rho)
    out["y"] = du
    return out


# the chain of the forward pass, the sums over a row twice more, and for the sums
# over the tokens one addition a row of a thread (at most 16 here) and the joins of
# 16 groups and 256 workgroups (16 at a time, then 16)
BACKWARD_STEPS = 3 * FORWARD_STEPS
SUM_STEPS = BACKWARD_STEPS + 64

BACKWARD = [case(T=T, H=H) for T, H in ((1, 2048), (3, 1), (5, 7), (40, 512), (17, 513), (600, 64),
                                        (9, 1025), (1029, 2048), (6, 4096), (5, 4097), (3, 8191))]
BACKWARD += [case(T=19, H=H, kind=k, dtype=d, gate=g, post=p, bias=b, offset=o, pad=pad)
             for (H, pad), (k, d), (g, p, b, o) in itertools.product(
                 ((264, 0), (777, 5), (2304, 8)),
                 (("rms", "bf16"), ("layer", "f32"), ("layer", "f16")),
                 (("none", False, False, False), ("token", True, True, True),
                  ("column", False, True, True), ("column", True, False, False)))]
BACKWARD += [case(dtype="f16", w_dtype="f32", H=1032), case(dtype="bf16", w_dtype="f32", H=2050),
             case(eps=0.0, T=18, H=100), case(scale=0.0), case(residual=False), case(T=4099, H=33)]


def grads_in(c, d, seed=1):
    g = torch.Generator().manual_seed(77 + seed)
    dt = R.TYPES[c["dtype"]][0]
    dev = [rows(torch.randn((c["T"], c["H"]), generator=g), c["pad"], dt) for _ in range(2)]
    return dev, [t.cpu().double()[:, :c["H"]] for t in dev]


@pytest.mark.parametrize("which", ["both", "dout", "dn"])
@pytest.mark.parametrize("c", BACKWARD, ids=name)
def test_backward(c, which):
    d, v = inputs(c)
    (dout, dn), (vo, vn) = grads_in(c, d)
    if which == "dout":
        dn = vn = None
    if which == "dn":
        dout = vo = None
    out = gradient_buffers(c, d, dn is not None)
    backward(c, d, dout, dn, out)
    torch.cuda.synchronize()
    want, size = reference(c, v, vo, vn), sizes(c, v, vo, vn)
    dt, H = R.TYPES[c["dtype"]][0], c["H"]
    for n, got in zip(NAMES, out):
        if got is None:
            continue
        w = want.get(n)
        summed = got.dim() == 1
        got, pad = (got, None) if summed else (got[:, :H], got[:, H:])
        check(got.reshape(w.shape), w, size[n].reshape(w.shape),
              SUM_STEPS if summed else BACKWARD_STEPS, torch.float32 if summed else dt, n)
        assert pad is None or (pad == -3.0).all()
    # any one of them alone: the same bits
    for i, got in enumerate(out):
        if got is not None:
            alone = [None] * 7
            alone[i] = torch.full_like(got, -3.0)
            backward(c, d, dout, dn, alone)
            assert torch.equal(alone[i], got), NAMES[i]


def test_backward_without_block():
    c = case(post=False, gate="none", bias=False, H=264, T=37, kind="layer")
    d, v = inputs(c)
    d["y"] = v["y"] = None
    (_, dn), (_, vn) = grads_in(c, d)
    out = [None, torch.empty_like(dn), None, None, None, torch.empty(264, device=DEV),
           torch.empty(264, device=DEV)]
    backward(c, d, None, dn, out)
    want, size = reference(c, v, None, vn), sizes(c, v, None, vn)
    check(out[1], want["residual"], size["residual"], BACKWARD_STEPS, torch.float16, "residual")
    check(out[5], want["pre_w"], size["pre_w"], SUM_STEPS, torch.float32, "pre_w")
    check(out[6], vn.sum(0), size["pre_b"], SUM_STEPS, torch.float32, "pre_b")


def test_backward_against_differences():
    """Each gradient along random directions against central differences of the
    64-bit definition; a difference's own error is bounded by the change that half
    the step makes (it falls with the square of the step)."""
    c = case(T=6, H=40, dtype="f32", kind="layer", gate="token", pad=0)
    d, v = inputs(c)
    (dout, dn), (vo, vn) = grads_in(c, d)
    out = gradient_buffers(c, d)
    backward(c, d, dout, dn, out)
    size = sizes(c, v, vo, vn)
    g = torch.Generator().manual_seed(5)

    def loss(w):
        r, n = R.block_norm_ref(c, w)
        return float((r * vo).sum() + (n * vn).sum())
    for key, got in zip(NAMES, out):
        e = torch.randn(v[key].shape, generator=g, dtype=torch.float64)
        slope = [(loss(dict(v, **{key: v[key] + h * e})) - loss(dict(v, **{key: v[key] - h * e})))
                 / (2 * h) for h in (1e-4, 5e-5)]
        own = float((got.cpu().double().reshape(e.shape) * e).sum())
        room = abs(slope[0] - slope[1]) + 1e-9 * abs(slope[0]) \
            + float((SUM_STEPS * R.U * size[key].reshape(e.shape) * e.abs()).sum())
        assert abs(own - slope[1]) <= room, (key, own, slope)


def test_backward_in_place():
    c = case(H=640, T=21, gate="token")
    d, _ = inputs(c)
    (dout, dn), _ = grads_in(c, d)
    out = gradient_buffers(c, d)
    backward(c, d, dout, dn, out)
    alias = list(out)
    alias[0], alias[1] = dn, dout
    alias[3:] = [torch.empty(640, device=DEV) for _ in range(4)]
    want = [t.clone() for t in out]
    backward(c, d, dout, dn, alias)
    for a, w in zip(alias, want):
        assert torch.equal(a, w)


# more rows than the workgroups' first turn takes: later turns' rows travel while the
# turn before is computed
TURNS = [case(T=3100, H=2048, bias=False, pad=8, gate="column"),
         case(T=2100, H=2000, bias=False, pad=0, gate="token", dtype="bf16", w_dtype="f32"),
         case(T=8300, H=264, bias=False, pad=8, gate="none", offset=True),
         case(T=1100, H=4096, bias=False, pad=0, post=False, gate="none", kind="layer"),
         case(T=2100, H=1024, bias=True, pad=0, gate="none", kind="layer", residual=False)]


@pytest.mark.parametrize("c", TURNS, ids=name)
def test_backward_turns(c):
    say("block norm backward, turns: " + name(c))
    d, v = inputs(c)
    (dout, dn), (vo, vn) = grads_in(c, d)
    out = gradient_buffers(c, d)
    backward(c, d, dout, dn, out)
    torch.cuda.synchronize()
    want, size = reference(c, v, vo, vn), sizes(c, v, vo, vn)
    for n, got in zip(NAMES, out):
        if got is None:
            continue
        w, summed = want[n], got.dim() == 1
        rest = None if summed else got[:, c["H"]:]
        got = got if summed else got[:, :c["H"]]
        check(got.reshape(w.shape), w, size[n].reshape(w.shape),
              SUM_STEPS if summed else BACKWARD_STEPS,
              torch.float32 if summed else R.TYPES[c["dtype"]][0], n)
        assert rest is None or (rest == -3.0).all()
    # any number of stores behind the loads, and over the rows that came in: the same bits
    for keep in ([], [0], [1], [2], [0, 1], [0, 2], [1, 2]):
        some = [torch.full_like(t, -3.0) if t is not None and (i in keep or i > 2) else None
                for i, t in enumerate(out)]
        backward(c, d, dout, dn, some)
        for a, b in zip(some, out):
            assert a is None or torch.equal(a, b)
    rows_in = [dn, dout][:2 if out[1] is not None else 1]
    over = rows_in + [None] * (7 - len(rows_in))
    backward(c, d, dout, dn, over)
    for a, b in zip(rows_in, out):
        assert torch.equal(a[:, :c["H"]], b[:, :c["H"]])


def test_backward_bad_rows_stay_alone():
    c = case(T=2100, H=2048, bias=False, pad=0, gate="token")
    d, _ = inputs(c)
    (dout, dn), _ = grads_in(c, d)
    good = [0, 1, 3, 1023, 1024, 1025, 2047, 2048, 2049, 2099]
    bad = [2, 1022, 1026, 2050]
    out, again = gradient_buffers(c, d), gradient_buffers(c, d)
    backward(c, d, dout, dn, out)
    d["y"][bad, 5], dn[bad, 9] = float("nan"), float("inf")
    backward(c, d, dout, dn, again)
    for a, b in zip(out[:3], again[:3]):
        assert torch.equal(a[good], b[good]) and not torch.isfinite(b[bad]).all()


def test_backward_no_rows():
    c = case(T=0, H=72)
    out = [None, None, torch.full((72,), 5.0, device=DEV)] + \
        [torch.full((72,), 5.0, device=DEV) for _ in range(4)]
    M.moe_block_norm_backward(None, 72, None, 72, None, 72, None, 72, None, 0, 1.0, None, None,
                              None, *common(c), *out)
    assert all((t == 0).all() for t in out[2:])


def test_streams_and_graph():
    """On a side stream, and captured: every replay on new inputs gives the eager
    call's bits, also when two graphs with workspaces of their own alternate."""
    c = case(T=300, H=1000, gate="column")
    say("block norm: side stream and graphs")
    d, _ = inputs(c)
    (dout, dn), _ = grads_in(c, d)

    def eager(e, go, gn):
        o, n, g = torch.empty_like(e["y"]), torch.empty_like(e["y"]), gradient_buffers(c, e)
        forward(c, e, o, n)
        backward(c, e, go, gn, g)
        return [o, n] + g
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = eager(d, dout, dn)
    torch.cuda.synchronize()
    o, n, g = torch.empty_like(d["y"]), torch.empty_like(d["y"]), gradient_buffers(c, d)
    forward(c, d, o, n, side)
    ws = backward(c, d, dout, dn, g, side)
    side.synchronize()
    for a, b in zip([o, n] + g, want):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):
        ws = torch.empty_like(ws)
        o, n, g = torch.empty_like(d["y"]), torch.empty_like(d["y"]), gradient_buffers(c, d)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            forward(c, d, o, n)
            backward(c, d, dout, dn, g, ws=ws)
        graphs.append((graph, [o, n] + g))
    for i in range(4):
        d["y"].copy_(torch.randn_like(d["y"]) + i)
        dn.copy_(torch.randn_like(dn))
        want = eager(d, dout, dn)
        graph, outs = graphs[i % 2]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
