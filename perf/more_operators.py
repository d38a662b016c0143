"""What is measured of the operators around a routed block: cases, inputs, the
operators in plain torch, the library's calls, and exact values in 64 bits.

Operators ("op" of a case):
  norm     the end of one block and the start of the next: u = post(y) (or y),
           r = residual + scale * gate * u, n = pre(r), with RMS or layer norms;
           with "grad" its backward pass
  linear   out = residual + act(x w^T + bias) of fp16 matrices; with "grad" the
           gradients of x, w and bias from those of out
  balance  per-expert counts, mean probabilities, balance loss and z loss of
           router logits over the unmasked tokens; with "grad" the gradient of
           the logits too
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode token between two blocks: the residual add and the pre-norm
        dict(name="norm_1x2048", op="norm", grad=False, T=1, H=2048, kind="rms", post=False,
             gate="none", scale=1.0, bias=False, offset=False, pad=0, type="f16"),
        # a ragged chunk of a narrow model: layer norms with biases, a gate per
        # token, rows that lie in a wider buffer
        dict(name="norm_333x1000", op="norm", grad=False, T=333, H=1000, kind="layer", post=True,
             gate="token", scale=0.5, bias=True, offset=False, pad=5, type="bf16"),
        # a prefill batch with norms on both sides of the block and a learned gate
        dict(name="norm_4096x2048", op="norm", grad=False, T=4096, H=2048, kind="rms", post=True,
             gate="column", scale=1.0, bias=False, offset=True, pad=0, type="f16"),
        # the backward pass of that batch
        dict(name="norm_backward_4096x2048", op="norm", grad=True, T=4096, H=2048, kind="rms",
             post=True, gate="column", scale=1.0, bias=False, offset=True, pad=0, type="f16"),
        # one decode token through a 5632 x 2048 projection
        dict(name="linear_1", op="linear", grad=False, M=1, N=5632, K=2048, act="silu", bias=True,
             residual=False, out="f16"),
        # a ragged batch through a small projection, added to its residual
        dict(name="linear_333", op="linear", grad=False, M=333, N=1408, K=2000, act="gelu",
             bias=True, residual=True, out="f16"),
        # a prefill batch through 11264 x 2048
        dict(name="linear_4096", op="linear", grad=False, M=4096, N=11264, K=2048, act="none",
             bias=False, residual=False, out="f16"),
        # the gradients of an activated projection of 4096 tokens
        dict(name="linear_backward_4096", op="linear", grad=True, M=4096, N=5632, K=2048,
             act="silu", bias=True, residual=False, out="f16"),
        # the gradients of a 64-expert router's fp32 logits: few columns, many rows
        dict(name="linear_backward_router", op="linear", grad=True, M=4096, N=64, K=2048,
             act="none", bias=True, residual=False, out="f32"),
        # the load of a few concurrent decode tokens over 64 experts
        dict(name="balance_16x64", op="balance", grad=False, T=16, E=64, k=8, score="softmax",
             masked=0.0, z=False, zipf=0.0, type="f32", gtype="f32"),
        # a ragged, padded training batch of the 60-expert layer
        dict(name="balance_777x60", op="balance", grad=True, T=777, E=60, k=4, score="softmax",
             masked=0.1, z=True, zipf=0.0, type="f16", gtype="f16"),
        # a training batch of the 512-expert layer with skewed load, sigmoid scores
        dict(name="balance_4096x512", op="balance", grad=True, T=4096, E=512, k=10,
             score="sigmoid", masked=0.0, z=True, zipf=1.1, type="f32", gtype="f32"),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "balance"])
    grad = rng.random() < 0.5
    if op == "norm":
        H = rng.choice([_logu(rng, 8, 8192), 8 * _logu(rng, 1, 1024)])
        return dict(op=op, grad=grad, T=_logu(rng, 1, min(16384, 4096 * 2048 // H)), H=H,
                    kind=rng.choice(["rms", "layer"]), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "column", "token"]), scale=rng.choice([1.0, 0.5]),
                    bias=rng.random() < 0.5, offset=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 3]),
                    type=rng.choice(["f16", "bf16", "f32"]) if H <= 4096 else "f16")
    if op == "linear":
        # the backward pass does twice the work
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
        return dict(op=op, grad=grad, M=_logu(rng, 1, 4096), N=_logu(rng, 16, 5632 if grad else 11264),
                    K=8 * _logu(rng, 4, 256), act=act, bias=rng.random() < 0.5,
                    residual=not grad and rng.random() < 0.5,
                    out=rng.choice(["f16", "f32"]) if not grad or act == "none" else "f16")
    E = _logu(rng, 4, 512)
    return dict(op=op, grad=grad, T=_logu(rng, 1, 4096), E=E, k=rng.randint(1, min(16, E)),
                score=rng.choice(["softmax", "sigmoid"]), masked=rng.choice([0.0, 0.1, 0.5]),
                z=rng.random() < 0.5, zipf=rng.choice([0.0, 1.1]),
                type=rng.choice(["f16", "bf16", "f32"]), gtype=rng.choice(["f16", "bf16", "f32"]))


# ----------------------------------------------------------------- inputs

EPS = 1e-5
COEF, ZCOEF = 0.01, 0.001


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(x, pad, dtype):
    """x as rows of a buffer that is `pad` elements wider."""
    wide = torch.zeros((x.shape[0], x.shape[1] + pad), dtype=dtype, device="cuda")
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def prepare(case, seed):
    c, g = dict(case), _generator(seed)
    st = {"case": c}
    if c["op"] == "norm":
        T, H, dt = c["T"], c["H"], TYPES[c["type"]]
        rows = lambda x: _rows(x, c["pad"], dt)  # noqa: E731
        st["y"], st["residual"] = rows(_randn(g, T, H)), rows(2.0 * _randn(g, T, H))
        base = 0.0 if c["offset"] else 1.0   # weights near one, or their distance from one
        weight = lambda: (base + 0.1 * _randn(g, H)).to(dt)  # noqa: E731
        st["pre_w"], st["post_w"] = weight(), weight() if c["post"] else None
        st["pre_b"] = (0.1 * _randn(g, H)).to(dt) if c["bias"] else None
        st["post_b"] = (0.1 * _randn(g, H)).to(dt) if c["bias"] and c["post"] else None
        st["gate"] = None
        if c["gate"] == "column":
            st["gate"] = (0.5 + 0.1 * _randn(g, 1, H)).to(dt)
        elif c["gate"] == "token":
            st["gate"] = rows(torch.sigmoid(_randn(g, T, H)))
        if c["grad"]:
            st["dout"], st["dn"] = rows(_randn(g, T, H)), rows(_randn(g, T, H))
        st["out"] = [rows(torch.zeros((T, H), device="cuda")) for _ in range(2)]
        if c["grad"]:
            st["dgate"] = None if st["gate"] is None else \
                torch.empty((1, H), device="cuda") if c["gate"] == "column" else \
                rows(torch.zeros((T, H), device="cuda"))
            st["dweights"] = [None if w is None else torch.empty(H, device="cuda")
                              for w in (st["post_w"], st["post_b"], st["pre_w"], st["pre_b"])]
    elif c["op"] == "linear":
        M, N, K, dt = c["M"], c["N"], c["K"], TYPES[c["out"]]
        e = lambda *s, t=dt: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        st["x"], st["w"] = _randn(g, M, K).half(), (0.02 * _randn(g, N, K)).half()
        st["bias"] = 0.1 * _randn(g, N) if c["bias"] else None
        st["residual"] = _randn(g, M, N).to(dt) if c["residual"] else None
        if c["grad"]:
            st["dy"] = _randn(g, M, N).half()
            st["z"] = None   # what the forward pass keeps, where the activation has need of it
            if c["act"] != "none":
                st["z"] = (st["x"].float() @ st["w"].float().t()
                           + (0.0 if st["bias"] is None else st["bias"])).half()
            st["out"] = (e(M, K), e(N, K), e(N, t=torch.float32) if c["bias"] else None)
        else:
            st["out"] = e(M, N)
    else:
        T, E, k = c["T"], c["E"], c["k"]
        l = 0.9 * _randn(g, T, E)
        if c["zipf"]:
            rank = torch.randperm(E, generator=g, device="cuda") + 1
            l = l - c["zipf"] * torch.log(rank.float())
        st["logits"] = l.to(TYPES[c["type"]])
        st["idx"] = torch.sort(st["logits"].float(), dim=1, descending=True,
                               stable=True)[1][:, :k].int().contiguous()
        st["mask"] = None    # 1: a token that counts, 0: padding
        if c["masked"]:
            keep = torch.rand(T, generator=g, device="cuda") >= c["masked"]
            st["mask"] = keep.to(torch.uint8)
        st["d_loss"] = torch.full((1,), 65536.0, device="cuda")    # the training's loss scale
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        st["out"] = (e(E, t=torch.int32), e(E), e(2)) + (
            (e(T, E, t=TYPES[c["gtype"]]),) if c["grad"] else ())
    return st


# ------------------------------------------------------------- plain forms

def _plain_stats(v, kind):
    """(v less its mean or v, reciprocal root) of the rows."""
    c = v - v.mean(dim=1, keepdim=True) if kind == "layer" else v
    return c, torch.rsqrt((c * c).mean(dim=1, keepdim=True) + EPS)


def _plain_weight(w, offset):
    return w.float() + 1.0 if offset else w.float()


def _plain_norm_forward(st):
    """(u, xhat and reciprocal root of the post norm, r, those of the pre norm), fp32."""
    c = st["case"]
    u, post = st["y"].float(), None
    if c["post"]:
        v, rho = _plain_stats(u, c["kind"])
        post = (v * rho, rho)
        u = post[0] * _plain_weight(st["post_w"], c["offset"])
        if st["post_b"] is not None:
            u = u + st["post_b"].float()
    gu = u if st["gate"] is None else st["gate"].float() * u
    r = st["residual"].float() + c["scale"] * gu
    v, rho = _plain_stats(r, c["kind"])
    return u, post, r, (v * rho, rho)


def _plain_norm(st):
    c, dt = st["case"], TYPES[st["case"]["type"]]
    u, post, r, pre = _plain_norm_forward(st)
    n = pre[0] * _plain_weight(st["pre_w"], c["offset"])
    if st["pre_b"] is not None:
        n = n + st["pre_b"].float()
    return r.to(dt), n.to(dt)


def _plain_norm_input_grad(dn, w, xhat, rho, kind):
    g = dn * w
    d = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(dim=1, keepdim=True)
    return rho * d


def _plain_norm_backward(st):
    c, dt = st["case"], TYPES[st["case"]["type"]]
    u, post, r, pre = _plain_norm_forward(st)
    dn = st["dn"].float()
    dr = st["dout"].float() + _plain_norm_input_grad(
        dn, _plain_weight(st["pre_w"], c["offset"]), *pre, c["kind"])
    du = c["scale"] * dr
    dgate = None
    if st["gate"] is not None:
        dgate = du * u
        dgate = dgate.sum(dim=0, keepdim=True) if c["gate"] == "column" else dgate.to(dt)
        du = du * st["gate"].float()
    dy, dpost = du, [None, None]
    if c["post"]:
        dpost = [(du * post[0]).sum(dim=0), None if st["post_b"] is None else du.sum(dim=0)]
        dy = _plain_norm_input_grad(du, _plain_weight(st["post_w"], c["offset"]), *post, c["kind"])
    dpre = [(dn * pre[0]).sum(dim=0), None if st["pre_b"] is None else dn.sum(dim=0)]
    return [t for t in [dy.to(dt), dr.to(dt), dgate] + dpost + dpre if t is not None]


def _plain_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) \
            + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    a = math.sqrt(2.0 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)


def _plain_linear(st):
    c, dt = st["case"], TYPES[st["case"]["out"]]
    if c["grad"]:
        dz = st["dy"].float()
        if c["act"] != "none":
            dz = dz * _plain_act_grad(st["z"].float(), c["act"])
        grads = [(dz @ st["w"].float()).to(dt), (dz.t() @ st["x"].float()).to(dt)]
        return grads + ([dz.sum(dim=0)] if c["bias"] else [])
    z = st["x"].float() @ st["w"].float().t()
    if st["bias"] is not None:
        z = z + st["bias"]
    out = _plain_act(z, c["act"])
    if st["residual"] is not None:
        out = out + st["residual"].float()
    return out.to(dt)


def _plain_balance(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = st["logits"].float()
    m = torch.ones(T, device="cuda") if st["mask"] is None else (st["mask"] != 0).float()
    counts = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add_(
        0, st["idx"].long().reshape(-1), m.long().repeat_interleave(k))
    n = m.sum().clamp_min(1.0)
    top = l.amax(dim=1, keepdim=True)
    ex = torch.exp(l - top)
    total = ex.sum(dim=1, keepdim=True)
    soft, lse = ex / total, (top + torch.log(total))[:, 0]
    s = 1.0 / (1.0 + torch.exp(-l))
    p = soft if c["score"] == "softmax" else s / s.sum(dim=1, keepdim=True)
    mean = (p * m[:, None]).sum(dim=0) / n
    f = counts.float() / counts.sum().clamp_min(1).float()
    z = ZCOEF if c["z"] else 0.0
    losses = torch.stack([COEF * E * (f * mean).sum(), z * (lse * lse * m).sum() / n])
    out = [counts.int(), mean, losses]
    if c["grad"]:
        # sum p = 1: f less 1 / E gives the same gradient, without its cancellation
        d = (counts.double() * E - counts.sum().double()).div(counts.sum().clamp_min(1)).float()
        dp = COEF / n * (d - (p * d).sum(dim=1, keepdim=True))
        dl = p * dp if c["score"] == "softmax" else p * (1.0 - s) * dp
        dl = dl + z * 2.0 / n * lse[:, None] * soft
        out.append((st["d_loss"] * m[:, None] * dl).to(TYPES[c["gtype"]]))
    return out


# ------------------------------------------------------ the library's calls

def _own_workspace(st, nbytes):
    """The caller's workspace of the state's operator, allocated once."""
    if "workspace" not in st:
        st["workspace"] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    return st["workspace"]


def _own_norm(st, M, types):
    c = st["case"]
    ld = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    gate, ldg = st["gate"], 0 if c["gate"] == "column" else ld(st["gate"])
    kind = M.MOE_NORM_RMS if c["kind"] == "rms" else M.MOE_NORM_LAYER
    flags = (M.MOE_NORM_POST if c["post"] else 0) | (M.MOE_NORM_UNIT_OFFSET if c["offset"] else 0)
    dt, (a, b) = types[c["type"]], st["out"]
    if not c["grad"]:
        M.moe_block_norm(st["y"], ld(st["y"]), st["residual"], ld(st["residual"]), gate, ldg,
                         c["scale"], st["post_w"], st["post_b"], st["pre_w"], st["pre_b"], dt, dt,
                         kind, flags, EPS, c["T"], c["H"], a, ld(a), b, ld(b))
        return st["out"]
    n = M.moe_block_norm_backward_workspace_bytes(c["T"], c["H"])
    M.moe_block_norm_backward(st["dout"], ld(st["dout"]), st["dn"], ld(st["dn"]),
                              st["y"], ld(st["y"]), st["residual"], ld(st["residual"]), gate, ldg,
                              c["scale"], st["post_w"], st["post_b"], st["pre_w"], dt, dt, kind,
                              flags, EPS, c["T"], c["H"], a, b, st["dgate"], *st["dweights"],
                              _own_workspace(st, n), n)
    return [t for t in [a, b, st["dgate"]] + st["dweights"] if t is not None]


def _own_linear(st, M, types):
    c = st["case"]
    m, n, k = c["M"], c["N"], c["K"]
    act = {"none": M.MOE_ACT_NONE, "relu": M.MOE_ACT_RELU, "silu": M.MOE_ACT_SILU,
           "gelu": M.MOE_ACT_GELU, "gelu_tanh": M.MOE_ACT_GELU_TANH}[c["act"]]
    if c["grad"]:
        dx, dw, db = st["out"]
        nb = M.moe_linear_f16_backward_workspace_bytes(m, n, k)
        M.moe_linear_f16_backward(st["dy"], n, st["z"], n, act, st["x"], k, st["w"], k, m, n, k,
                                  dx, k, dw, k, types[c["out"]], db, _own_workspace(st, nb), nb)
        return [t for t in st["out"] if t is not None]
    nb = M.moe_linear_f16_workspace_bytes(m, n, k)
    M.moe_linear_f16(st["x"], k, st["w"], k, st["bias"], act, st["residual"], n, m, n, k,
                     st["out"], types[c["out"]], n, None, 0, _own_workspace(st, nb), nb)
    return st["out"]


def _own_balance(st, M, types):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    counts, mean, losses = st["out"][:3]
    score = M.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else M.MOE_SCORE_SIGMOID
    nb = M.moe_balance_loss_workspace_bytes(T, E)
    grad = (st["out"][3], types[c["gtype"]], E) if c["grad"] else (None, M.MOE_DTYPE_F32, E)
    M.moe_balance_loss(st["logits"], types[c["type"]], E, st["idx"], st["mask"], T, E, k, score,
                       COEF, ZCOEF if c["z"] else 0.0, counts, mean, losses, st["d_loss"], *grad,
                       _own_workspace(st, nb), nb)
    return list(st["out"])


def run(state):
    op = state["case"]["op"]
    if own:
        import int4_weight_only_router_amd as M
        types = {"f16": M.MOE_DTYPE_F16, "bf16": M.MOE_DTYPE_BF16, "f32": M.MOE_DTYPE_F32}
        return {"norm": _own_norm, "linear": _own_linear, "balance": _own_balance}[op](
            state, M, types)
    if op == "norm":
        return _plain_norm_backward(state) if state["case"]["grad"] else _plain_norm(state)
    return _plain_linear(state) if op == "linear" else _plain_balance(state)


def work(case):
    c = case
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if c["op"] == "norm":
        T, H, s = c["T"], c["H"], size[c["type"]]
        token_gate = c["gate"] == "token"
        rows = 4 + token_gate + c["grad"] * (2 + token_gate)
        vectors = 1 + c["post"] + c["bias"] * (1 + c["post"]) + (c["gate"] == "column")
        return {"bytes": rows * T * H * s + vectors * H * (s + 4 * c["grad"]),
                "flops": (40 if c["grad"] else 16) * T * H}
    if c["op"] == "linear":
        M, N, K, s = c["M"], c["N"], c["K"], size[c["out"]]
        if c["grad"]:
            return {"bytes": 2 * (M * N * (2 if c["act"] != "none" else 1) + M * K + N * K)
                    + s * (M * K + N * K) + 4 * N * c["bias"], "flops": 4 * M * N * K}
        return {"bytes": 2 * (M + N) * K + M * N * s * (1 + c["residual"]) + 4 * N * c["bias"],
                "flops": 2 * M * N * K}
    T, E, k = c["T"], c["E"], c["k"]
    return {"bytes": T * E * (size[c["type"]] + (size[c["gtype"]] if c["grad"] else 0)) + 4 * T * k
            + (T if c["masked"] else 0) + 8 * E + 8, "flops": (30 if c["grad"] else 15) * T * E}


# ------------------------------------------------------- exact, in 64 bits

def _exact_norm(st):
    """The definition in 64 bits; gradients by differentiating it."""
    c = st["case"]
    leaf = {k: st[k].detach().double().clone().requires_grad_(c["grad"])
            for k in ("y", "residual", "gate", "post_w", "post_b", "pre_w", "pre_b")
            if st.get(k) is not None}

    def norm(v, w, b):
        if c["kind"] == "layer":
            var, mean = torch.var_mean(v, dim=-1, unbiased=False, keepdim=True)
            v = (v - mean) / torch.sqrt(var + EPS)
        else:
            v = v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS)
        v = v * (1 + leaf[w] if c["offset"] else leaf[w])
        return v + leaf[b] if b in leaf else v

    u = norm(leaf["y"], "post_w", "post_b") if c["post"] else leaf["y"]
    r = torch.addcmul(leaf["residual"], u, leaf["gate"] if "gate" in leaf else torch.ones_like(u),
                      value=c["scale"])
    n = norm(r, "pre_w", "pre_b")
    if not c["grad"]:
        return r, n
    order = [k for k in ("y", "residual", "gate", "post_w", "post_b", "pre_w", "pre_b") if k in leaf]
    return list(torch.autograd.grad([r, n], [leaf[k] for k in order],
                                    [st["dout"].double(), st["dn"].double()]))


def _exact_act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * (1.0 - 0.5 * torch.erfc(z / 2.0 ** 0.5))
    if act == "gelu_tanh":   # (1 + tanh a) / 2 is the logistic function of 2 a
        return z * torch.sigmoid((8.0 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return z


def _exact_linear(st):
    c = st["case"]
    x, w = st["x"].double(), st["w"].double()
    if c["grad"]:
        dz = st["dy"].double()
        if c["act"] != "none":
            z = st["z"].double().requires_grad_(True)
            dz, = torch.autograd.grad(_exact_act(z, c["act"]), z, dz)
        return [torch.matmul(dz, w), torch.matmul(dz.t(), x)] + (
            [dz.sum(dim=0)] if c["bias"] else [])
    z = torch.matmul(x, w.t())
    if c["bias"]:
        z += st["bias"].double()
    out = _exact_act(z, c["act"])
    return out + st["residual"].double() if c["residual"] else out


def _exact_balance(st):
    c = st["case"]
    T, E = c["T"], c["E"]
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"] > 0
    l = st["logits"].double()[keep].requires_grad_(c["grad"])
    counts = torch.bincount(st["idx"][keep].reshape(-1).long(), minlength=E)
    share = counts.double() / max(1, int(counts.sum()))
    rows = max(1, l.shape[0])
    log_s = torch.log_softmax(l, dim=1) if c["score"] == "softmax" else \
        torch.log_softmax(torch.nn.functional.logsigmoid(l), dim=1)
    mean = torch.exp(log_s).sum(dim=0) / rows
    balance = COEF * E * torch.dot(share, mean)
    z = (ZCOEF if c["z"] else 0.0) * torch.logsumexp(l, dim=1).pow(2).sum() / rows
    out = [counts.int(), mean.detach(), torch.stack([balance, z]).detach()]
    if c["grad"]:
        d = torch.zeros((T, E), dtype=torch.float64, device="cuda")
        d[keep], = torch.autograd.grad(balance + z, l, st["d_loss"].double()[0])
        out.append(d)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "balance": _exact_balance}[
        st["case"]["op"]](st)
