"""64-bit forms of the operators around a routed block, their gradients by
differentiation, and how far an fp32 kernel may be from them.

U is fp32's half step.  Sizes of intermediate values are formed with every term
in magnitude, so that a bound holds where terms cancel too."""
import numpy as np
import torch

import int4_weight_only_router_amd as M

U = 2.0 ** -24
TYPES = {"f16": (torch.float16, M.MOE_DTYPE_F16), "bf16": (torch.bfloat16, M.MOE_DTYPE_BF16),
         "f32": (torch.float32, M.MOE_DTYPE_F32)}


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the smallest step of the type: rounding near zero."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps


# ------------------------------------------------------------------- norms

def norm_ref(v, w, b, kind, eps, offset):
    if kind == "layer":
        v = v - v.mean(dim=-1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(dim=-1, keepdim=True) + eps)
    if w is not None:
        v = v * (w + 1.0 if offset else w)
    return v if b is None else v + b


def block_norm_ref(c, t):
    """(r, n) of the case's 64-bit tensors t (a dict; absent ones None)."""
    u = t["y"]
    if u is not None:
        if c["post"]:
            u = norm_ref(u, t["post_w"], t["post_b"], c["kind"], c["eps"], c["offset"])
        if t["gate"] is not None:
            u = t["gate"] * u
        u = c["scale"] * u
    r = t["residual"] if u is None else u if t["residual"] is None else t["residual"] + u
    return r, norm_ref(r, t["pre_w"], t["pre_b"], c["kind"], c["eps"], c["offset"])


def _norm_size(v, size, w, b, kind, eps, offset):
    """Size of a norm's output per element where its input v is off by up to
    `size` (in units of U times a constant): the input's own, what the mean and
    the root take from it, the weight and the bias."""
    if kind == "layer":
        size = size + size.mean(dim=-1, keepdim=True)
        v = v - v.mean(dim=-1, keepdim=True)
    rho = 1.0 / torch.sqrt((v * v).mean(dim=-1, keepdim=True) + eps)
    m = v * rho
    # d m = rho (d v - m mean(m d v)), plus m's own roundings
    out = rho * size + m.abs() * (1.0 + rho * (m.abs() * size).mean(dim=-1, keepdim=True))
    if w is not None:
        out = out * (w + 1.0 if offset else w).abs()
    return out if b is None else out + b.abs()


def block_norm_sizes(c, t):
    """Sizes of r and n."""
    z = 0.0
    if t["y"] is not None:
        u, size = t["y"], torch.zeros_like(t["y"])
        if c["post"]:
            args = (t["post_w"], t["post_b"], c["kind"], c["eps"], c["offset"])
            size = _norm_size(u, u.abs(), *args)
            u = norm_ref(u, *args)
        size = size + u.abs()
        g = 1.0 if t["gate"] is None else t["gate"].abs()
        z = abs(c["scale"]) * g * size
    r = block_norm_ref(c, t)[0]
    sr = r.abs() + z + (0.0 if t["residual"] is None else t["residual"].abs())
    return sr, _norm_size(r, sr, t["pre_w"], t["pre_b"], c["kind"], c["eps"], c["offset"])


# -------------------------------------------------------------- activations

ACTS = {"none": M.MOE_ACT_NONE, "relu": M.MOE_ACT_RELU, "silu": M.MOE_ACT_SILU,
        "gelu": M.MOE_ACT_GELU, "gelu_tanh": M.MOE_ACT_GELU_TANH}


def act_ref(z, act):
    if act == "relu":
        return torch.relu(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * (1.0 - 0.5 * torch.erfc(z / 2.0 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def act_grad_ref(z, act):
    z = z.clone().requires_grad_(True)
    g, = torch.autograd.grad(act_ref(z, act).sum(), z)
    return g


# ------------------------------------------------------------------ balance

def balance_ref(logits, idx, mask, E, score, coef, zcoef, up=1.0):
    """counts, mean probabilities, losses, gradient, in 64 bits on the CPU; logits
    may hold -inf and NaN (masked experts)."""
    T = logits.shape[0]
    on = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    ids = idx[on].reshape(-1).long()
    counts = torch.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
    l0 = logits.double()
    l0 = torch.where(torch.isnan(l0), torch.full_like(l0, -np.inf), l0)
    l0 = l0.clamp_max(torch.finfo(torch.float32).max)
    n, total = int(on.sum()), max(1, int(counts.sum()))
    f = counts.double() / total
    grad, mean = torch.zeros_like(l0), torch.zeros(E, dtype=torch.float64)
    bal = z = 0.0
    for t in range(T):
        e = torch.isfinite(l0[t])
        if not on[t] or not e.any():
            continue
        l = l0[t][e].clone().requires_grad_(True)
        logs = l if score == M.MOE_SCORE_SOFTMAX else torch.nn.functional.logsigmoid(l)
        p = torch.softmax(logs, 0)
        b = coef * E / n * (f[e] * p).sum()
        zz = zcoef / n * torch.logsumexp(l, 0) ** 2
        g, = torch.autograd.grad(b + zz, l)
        grad[t][e] = up * g
        mean[e] += p.detach() / n
        bal, z = bal + float(b.detach()), z + float(zz.detach())
    return counts, mean, np.array([bal, z]), grad
