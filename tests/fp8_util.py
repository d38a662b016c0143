"""64-bit references of the FP8 and score-routing operators (numpy, written
from the formulas of the header)."""
import numpy as np
import torch

U32 = 2.0 ** -24          # half a step of fp32
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: U32}


def blocks(n):
    return (n + 127) // 128


def e4m3(v):
    """Nearest e4m3 value of each |v| <= 448, ties to even."""
    v = np.asarray(v, np.float64)
    e = np.maximum(np.frexp(v)[1] - 1, -6)
    step = np.ldexp(1.0, e - 3)
    return np.rint(v / step) * step


def e4m3_step(v):
    """Distance of neighbouring e4m3 values around v."""
    return np.ldexp(1.0, np.maximum(np.frexp(np.asarray(v, np.float64))[1] - 1, -6) - 3)


def scale_of(amax, pow2):
    """fp32 scale of a block of largest magnitude amax (fp32 array)."""
    amax = np.asarray(amax, np.float32)
    s = np.maximum(amax / np.float32(448), np.float32(2.0 ** -126))
    if pow2:
        b = s.view(np.uint32)
        s = np.where(b & 0x7fffff, (b & 0x7f800000) + 0x800000, b).astype(np.uint32).view(np.float32)
    return np.where(amax > 0, s, np.float32(0)).astype(np.float32)


def quantize(x, block, pow2):
    """(values of the codes, fp32 scales) of fp32 x [R, C]."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    rb, kb = -(-R // block), blocks(C)
    p = np.zeros((rb * block, kb * 128), np.float32)
    p[:R, :C] = x
    p = p.reshape(rb, block, kb, 128)
    s = scale_of(np.abs(p).max(axis=(1, 3)), pow2)
    d = np.where(s > 0, s, np.float32(1))
    q = e4m3((p / d[:, None, :, None]).astype(np.float32)).reshape(rb * block, kb * 128)
    return q[:R, :C], s


def spread(s, block, R, C):
    """Scales [.., R/block, C/128] repeated over their blocks, fp64 [R, C]."""
    return np.repeat(np.repeat(s.astype(np.float64), block, 0)[:R], 128, 1)[:, :C]


# the fp8 matrix instruction adds runs of eight neighbouring products on a grid
# of 13 bits below the run's largest: another product loses at most this of it
GRID = 2.0 ** -13


def product(xq, xs, wq, ws, runs=False):
    """(y, bound): the product in 64 bits and how far fp32 block sums may be
    off.  A block's 128 products are exact in fp32 (4 + 4 significant bits);
    their sum takes at most 128 roundings of at most a whole step (2 U32, in
    case the adder truncates) of the absolute sum, the scale product one, the
    accumulation one fma per block.  runs: the fp8 matrix instruction; seven of
    a run's products lose at most GRID of its largest each, and the largest of
    a run is at most the run's sum of |products|."""
    x = xq * spread(xs, 1, *xq.shape)
    w = wq * spread(ws, 128, *wq.shape)
    nkb = blocks(xq.shape[1])
    return x @ w.T, ((256 + nkb + 4) * U32 + runs * 7 * GRID) * (np.abs(x) @ np.abs(w).T)


def codes(t):
    """fp64 values of an e4m3 tensor."""
    return t.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)


def select(logits, bias, k, score, n_group, keep, top2, renorm, scale):
    """(idx, w) row by row."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    live = l > -np.inf
    l = np.where(live, np.minimum(l, float(np.finfo(np.float32).max)), 0.0)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    n = E // n_group
    idx = np.zeros((T, k), np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        s = np.zeros(E)
        a = live[t]
        if a.any():
            if score == "softmax":
                s[a] = np.exp(l[t, a] - l[t, a].max())
                s /= s.sum()
            else:
                with np.errstate(over="ignore"):
                    s[a] = 1.0 / (1.0 + np.exp(-l[t, a]))
        c = s + b
        rank = []
        for g in range(n_group):
            m = np.sort(c[g * n:(g + 1) * n][a[g * n:(g + 1) * n]])[::-1]
            rank.append(-np.inf if not m.size else m[:2 if top2 else 1].sum())
        kept = sorted(range(n_group), key=lambda g: (-rank[g], g))[:keep]
        pool = [e for g in kept for e in range(g * n, (g + 1) * n)]
        pool.sort(key=lambda e: (not a[e], -c[e] if a[e] else 0.0, e))
        idx[t] = pool[:k]
        v = s[idx[t]]
        if renorm:
            v = v / v.sum() if v.sum() > 0 else np.zeros(k)
        w[t] = v * np.float64(np.float32(scale))
    return idx, w


def grouping(idx, E):
    flat = idx.reshape(-1)
    counts = np.bincount(flat, minlength=E)
    perm = np.argsort(flat, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(flat.size)
    return counts, np.concatenate([[0], counts.cumsum()]), perm, inv


def experts_row(x, wg, wu, wd):
    """One expert on rows x (fp32 [n, H]); w*: (codes, scales).  Returns (y,
    bound) in 64 bits.

    g and u are off by product()'s bound; silu(g) u by their propagation plus
    (|g| + 8) 2 U32 relative (hardware exp2 and reciprocal, about one step
    each, and the rounded exponent).  An element of h whose error reaches the
    middle between two codes may take the other one: one step; if a block's
    largest magnitude may cross a power of two times 448, every element of the
    block may move by a step of the coarser scale."""
    xq, xs = quantize(x, 1, True)
    g, dg = product(xq, xs, *wg)
    u, du = product(xq, xs, *wu)
    sg = 1.0 / (1.0 + np.exp(-g))
    h = g * sg * u
    # |d silu / dg| <= 1.1
    dh = 1.1 * dg * np.abs(u) + np.abs(g * sg) * du + 1.1 * dg * du \
        + np.abs(h) * (np.abs(g) + 8) * 2 * U32
    n, I = h.shape
    kb = blocks(I)
    hq = np.zeros_like(h)
    hs = np.zeros((n, kb), np.float32)
    move = np.zeros_like(h)                 # how far a quantised value may be off
    for j in range(kb):
        c = slice(128 * j, min(I, 128 * j + 128))
        top = np.abs(h[:, c]).max(1)
        d = dh[:, c].max(1)
        s = scale_of(top.astype(np.float32), True).astype(np.float64)
        lo = scale_of(np.maximum(top - d, 0).astype(np.float32), True)
        hi = scale_of((top + d).astype(np.float32), True)
        hs[:, j] = s
        z = np.where(s > 0, s, 1.0)[:, None]
        v = h[:, c] / z
        hq[:, c] = e4m3(np.clip(v, -448, 448))
        step = e4m3_step(np.abs(v) + dh[:, c] / z)
        edge = np.abs(np.abs(v - hq[:, c]) - step / 2) <= dh[:, c] / z + step * 1e-6
        near = np.abs(np.abs(v - hq[:, c]) - step / 4) <= dh[:, c] / z + step * 1e-6
        flip = np.where(edge | near, step, 0.0)
        flip = np.where((lo != hi)[:, None], 2 * step, flip)
        move[:, c] = flip * z
    y, dy = product(hq, hs, *wd, runs=True)
    w = np.abs(wd[0] * spread(wd[1], 128, *wd[0].shape))
    return y, dy * 1.01 + move @ w.T
