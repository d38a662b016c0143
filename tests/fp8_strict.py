"""A bound on the L2 error of the FP8 experts' rows that wrong results do not
fit in at the sizes of real layers (the element bounds of fp8_util add every
possible step of h in absolute value, and grow past the result there)."""
import numpy as np

from tests import fp8_util as R

SWIGLU = 2 * R.U32   # hardware exp2 and reciprocal: about one step each, (|g| + 8) of them


def swiglu_error(g, u, dg, du):
    """How far silu(g) u may be off for g, u off by dg, du (|d silu / dg| <= 1.1)."""
    sg = 1.0 / (1.0 + np.exp(-g))
    return (1.1 * dg * np.abs(u) + np.abs(g * sg) * du + 1.1 * dg * du
            + np.abs(g * sg * u) * (np.abs(g) + 8) * SWIGLU)


def experts_l2(x, wg, wu, wd, runs):
    """(y, allowed): one expert on fp32 rows x in 64 bits, and the largest L2
    error of each fp16 row of y.

    h may be off by what fp32 sums leave (fp8_util.product).  A code of h then
    differs only where that error reaches the middle between two codes: f, one
    step there and zero elsewhere (two of the coarser block's steps throughout a
    block whose scale may differ).  The row of y moves by Wd f, in L2 at most
    the spectral norm of Wd's columns under f times |f|.  To that come the down
    product's error (runs: of the FP8 matrix instruction, fp8_util.product's
    bound replaced by its root mean square over a row: seven losses of a run,
    each below GRID of its largest product, of random sign and a third of their
    largest square on average) and the rounding to fp16."""
    xq, xs = R.quantize(x, 1, True)
    g, dg = R.product(xq, xs, *wg)
    u, du = R.product(xq, xs, *wu)
    h = g / (1.0 + np.exp(-g)) * u
    dh = swiglu_error(g, u, dg, du)
    n, I = h.shape
    hq, hs, f = np.zeros_like(h), np.zeros((n, R.blocks(I)), np.float32), np.zeros_like(h)
    for j in range(R.blocks(I)):
        c = slice(128 * j, min(I, 128 * j + 128))
        top, d = np.abs(h[:, c]).max(1), dh[:, c].max(1)
        hs[:, j] = R.scale_of(top.astype(np.float32), True)
        lo = R.scale_of(np.maximum(top - d, 0).astype(np.float32), True)
        hi = R.scale_of((top + d).astype(np.float32), True)
        z = np.where(hs[:, j] > 0, hs[:, j].astype(np.float64), 1.0)[:, None]
        v, dv = h[:, c] / z, dh[:, c] / z
        hq[:, c] = R.e4m3(np.clip(v, -448, 448))
        same = R.e4m3(np.clip(np.abs(v) - dv, 0, 448)) == R.e4m3(np.clip(np.abs(v) + dv, 0, 448))
        step = R.e4m3_step(np.abs(v) + dv)
        f[:, c] = np.where((lo != hi)[:, None], 2 * step, np.where(same, 0.0, step)) * z
    y, dy = R.product(hq, hs, *wd)
    w = wd[0] * R.spread(wd[1], 128, *wd[0].shape)
    allowed = np.sqrt(np.square(dy).sum(1))
    if runs:
        hv = hq * R.spread(hs, 1, n, I)
        allowed += np.sqrt(7 / 3) * R.GRID * np.sqrt((np.square(hv) @ np.square(w).T).sum(1))
    for r in range(n):
        s = np.flatnonzero(f[r])
        if s.size:
            top = np.linalg.eigvalsh(w[:, s].T @ w[:, s])[-1]
            allowed[r] += np.sqrt(max(top, 0.0)) * np.linalg.norm(f[r, s])
    half = 2.0 ** -11 * np.linalg.norm(y, axis=1) + 2.0 ** -25 * np.sqrt(y.shape[1])
    return y, 1.001 * allowed + half
