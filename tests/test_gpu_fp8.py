"""Block-scaled FP8 operators on the GPU against 64-bit references: codes and
scales equal, products and experts within bounds derived from fp32 sums of
128-long blocks (fp8_util)."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
from tests import fp8_util as R
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
TYPES = {"f32": (torch.float32, M.MOE_DTYPE_F32), "f16": (torch.float16, M.MOE_DTYPE_F16),
         "bf16": (torch.bfloat16, M.MOE_DTYPE_BF16)}


def _rand8(r, rows, cols, ld=None):
    """e4m3 bytes [rows, ld] on the device (NaN codes between the rows) and values."""
    ld = cols if ld is None else ld
    v = R.e4m3(np.clip(r.normal(0, 60, (rows, cols)), -448, 448))
    buf = torch.full((rows, ld), 0x7F, dtype=torch.uint8, device=DEV)
    buf[:, :cols] = torch.from_numpy(v.astype(np.float32)).to(F8).view(torch.uint8).to(DEV)
    return buf, v


# -------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,cols,block,ldx,ldq", [
    (1, 1, 1, 1, 1), (1, 2048, 1, 2048, 2048), (3, 130, 1, 130, 130), (5, 128, 1, 136, 144),
    (7, 1000, 1, 1003, 1001), (67, 1408, 1, 1408, 1408), (1, 1, 128, 1, 1),
    (130, 257, 128, 257, 257), (200, 256, 128, 264, 272), (127, 8, 128, 9, 8)])
def test_quantize(rows, cols, block, ldx, ldq, pow2, dtype):
    say("quantize %dx%d block=%d ld=%d/%d pow2=%d %s" % (rows, cols, block, ldx, ldq, pow2, dtype))
    tt, dt = TYPES[dtype]
    r = np.random.default_rng(rows * 7 + cols)
    x = torch.full((rows, ldx), float("nan"), dtype=tt)
    v = r.normal(0, 1, (rows, cols)) * np.exp(r.normal(0, 3, (rows, 1)))
    x[:, :cols] = torch.from_numpy(np.clip(v, -6e4, 6e4)).to(tt)
    if rows > 2:
        x[1, :cols] = 0.0                                     # a block of zeros
        x[2, :cols] = float(torch.finfo(tt).tiny) * 2.0 ** -3 if dtype == "f32" else 6e-8
    q = torch.full((rows, ldq), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((-(-rows // block) * R.blocks(cols) + 1,), -7.0, device=DEV)
    M.moe_quantize_fp8(x.to(DEV), dt, ldx, rows, cols, block, M.MOE_SCALE_POW2 if pow2 else 0, q,
                       ldq, s)
    torch.cuda.synchronize()
    rq, rs = R.quantize(x[:, :cols].float().numpy(), block, pow2)
    assert np.array_equal(s[:-1].cpu().numpy().view(np.uint32), rs.reshape(-1).view(np.uint32))
    assert float(s[-1]) == -7.0
    assert np.array_equal(R.codes(q)[:, :cols], rq)
    assert bool((q[:, cols:] == 0x55).all())


def test_quantize_every_value():
    """Every finite fp16 value, each in a block whose largest value is 448:
    the codes are the nearest e4m3 values, ties to even."""
    say("quantize every value")
    a = np.arange(65536, dtype=np.uint16).view(np.float16)
    a = a[np.isfinite(a.astype(np.float32)) & (np.abs(a.astype(np.float32)) <= 448)]
    n = -(-a.size // 127)
    x = np.zeros((n, 128), np.float16)
    x[:, 0] = 448
    x[:, 1:].reshape(-1)[:] = 0
    flat = np.zeros(n * 127, np.float16)
    flat[:a.size] = a
    x[:, 1:] = flat.reshape(n, 127)
    q = torch.empty((n, 128), dtype=torch.uint8, device=DEV)
    s = torch.empty(n, device=DEV)
    M.moe_quantize_fp8(torch.from_numpy(x).to(DEV), M.MOE_DTYPE_F16, 128, n, 128, 1,
                       M.MOE_SCALE_POW2, q, 128, s)
    assert bool((s == 1.0).all())
    assert np.array_equal(R.codes(q), R.e4m3(x.astype(np.float64)))


def test_quantize_non_finite():
    """A NaN or an infinity stays visible in the products with its block."""
    say("quantize non-finite")
    x = torch.ones((3, 256), dtype=torch.float32, device=DEV)
    x[0, 3] = float("nan")
    x[1, 200] = float("inf")
    for flags in (0, M.MOE_SCALE_POW2):
        q = torch.empty((3, 256), dtype=torch.uint8, device=DEV)
        s = torch.empty((3, 2), device=DEV)
        M.moe_quantize_fp8(x, M.MOE_DTYPE_F32, 256, 3, 256, 1, flags, q, 256, s)
        v = q.view(F8).float() * s.repeat_interleave(128, 1)
        assert bool(v[0, 3].isnan()) and not bool(v[0, 128:].isnan().any())
        assert not bool(v[1, 200].isfinite()) and not bool(v[1, :128].isnan().any())
        assert bool(v[2].isfinite().all())


def test_quantize_more_rows_than_a_launch():
    """2^28 + 5 rows of one column: more than one launch."""
    say("quantize many rows")
    n = (1 << 28) + 5
    x = torch.randint(-3, 4, (n,), dtype=torch.int8, device=DEV).to(torch.float16)
    q = torch.full((n,), 9, dtype=torch.uint8, device=DEV)
    s = torch.full((n,), -1.0, device=DEV)
    M.moe_quantize_fp8(x, M.MOE_DTYPE_F16, 1, n, 1, 1, 0, q, 1, s)
    # a lone value takes the largest code, and 448 s gives it back
    code = torch.where(x > 0, 0x7E, 0).to(torch.uint8) + torch.where(x < 0, 0xFE, 0).to(torch.uint8)
    want = torch.from_numpy(np.arange(4, dtype=np.float32) / np.float32(448)).to(DEV)
    wrong = (q != code).sum() + (s != want[x.abs().int()]).sum()
    assert wrong.item() == 0


def test_quantize_far_rows():
    """Rows whose element offsets pass 32 bits."""
    say("quantize far rows")
    ld = (1 << 30) + 8
    x = torch.empty(2 * ld + 128 + ld, dtype=torch.float16, device=DEV)
    q = torch.empty(4, dtype=torch.uint8, device=DEV)
    rows = torch.randn((4, 128), device=DEV).half()
    for i in range(3):
        x[i * ld:i * ld + 128] = rows[i]
    q = torch.empty((3, 128), dtype=torch.uint8, device=DEV)
    s = torch.empty(3, device=DEV)
    M.moe_quantize_fp8(x, M.MOE_DTYPE_F16, ld, 3, 128, 1, 0, q, 128, s)
    rq, rs = R.quantize(rows[:3].float().cpu().numpy(), 1, False)
    assert np.array_equal(s.cpu().numpy(), rs.reshape(-1)) and np.array_equal(R.codes(q), rq)


# ------------------------------------------------------------------ products

def _product(M_, N, K, dtype, ldx=None, ldw=None, ldo=None, seed=0):
    r = np.random.default_rng(M_ * 31 + N * 7 + K + seed)
    ldx, ldw, ldo = ldx or K, ldw or K, ldo or N
    xb, xv = _rand8(r, M_, K, ldx)
    wb, wv = _rand8(r, N, K, ldw)
    nkb = R.blocks(K)
    xs = np.exp(r.normal(-6, 1, (M_, nkb))).astype(np.float32)
    ws = np.exp(r.normal(-6, 1, (R.blocks(N), nkb))).astype(np.float32)
    tt, dt = TYPES[dtype]
    out = torch.full((M_ + 1, ldo), -7.0, dtype=tt, device=DEV)
    M.moe_gemm_fp8(xb, ldx, torch.from_numpy(xs).to(DEV), wb, ldw, torch.from_numpy(ws).to(DEV),
                   M_, N, K, out, dt, ldo)
    torch.cuda.synchronize()
    y, bound = R.product(xv, xs, wv, ws, runs=dtype != "f32")
    got = out[:M_, :N].double().cpu().numpy()
    half = R.HALF_STEP[tt]
    tol = bound + half * (np.abs(y) + bound)
    if dtype == "f16":
        tol = tol + 2.0 ** -25
    off = np.abs(got - y) - tol
    assert np.all(off <= 0), "off by %g over the bound at %s" % (
        off.max(), np.unravel_index(off.argmax(), off.shape))
    # over many outputs the errors are not all at their bound: the output's own
    # rounding and, of a run's seven losses below GRID of its largest, each of
    # its product's random sign and a third of its greatest square on average,
    # sqrt(7 / 3) GRID of the root sum of squares of the runs' largest products,
    # which is at most that of all products
    rms = np.sqrt((np.square(xv * R.spread(xs, 1, *xv.shape)) @
                   np.square(wv * R.spread(ws, 128, *wv.shape)).T).mean())
    assert np.sqrt(np.square(got - y).mean()) <= half * np.sqrt(np.square(y).mean()) \
        + np.sqrt(7 / 3) * R.GRID * rms
    assert bool((out[:M_, N:] == -7.0).all()) and bool((out[M_] == -7.0).all())


SHAPES = [(1, 1, 16), (1, 32, 128), (1, 5632, 2048), (3, 33, 48), (16, 100, 192), (17, 130, 144),
          (33, 64, 2048), (64, 257, 1040), (65, 31, 80), (333, 1408, 2000), (100, 2048, 4096)]
TILES = [(1600, 4000, 64), (1531, 4117, 400), (4096, 1536, 256), (130, 24700, 144),
         (1000, 1500, 272), (700, 5000, 144), (2500, 5000, 80), (2000, 9000, 48)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k, dtype):
    say("product %dx%dx%d %s" % (m, n, k, dtype))
    _product(m, n, k, dtype)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("m,n,k", TILES)
def test_product_tiles(m, n, k, dtype):
    say("product tiles %dx%dx%d" % (m, n, k))
    _product(m, n, k, dtype)


@pytest.mark.parametrize("m,n,k,ldx,ldw,ldo", [(5, 40, 96, 112, 128, 41), (70, 130, 272, 288, 304,
                                               133), (1600, 4001, 144, 160, 176, 4003),
                                               (1600, 4000, 144, 160, 176, 4004)])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_product_strides(m, n, k, ldx, ldw, ldo, dtype):
    """NaN codes lie between the rows: a byte read past K would show."""
    say("product strides %dx%dx%d %d/%d/%d" % (m, n, k, ldx, ldw, ldo))
    _product(m, n, k, dtype, ldx, ldw, ldo)


@pytest.mark.parametrize("m,n,k,dtype,ldx,ldw,ldo", [
    (20, 40, 144, "f32", 1 << 27, 1 << 27, (1 << 27) + 1),
    (1500, 1500, 144, "f16", 1 << 21, 1 << 21, 1 << 21)])
def test_product_far_rows(m, n, k, dtype, ldx, ldw, ldo):
    """Rows whose offsets pass 32 bits, in both kernels."""
    say("product far rows %dx%dx%d" % (m, n, k))
    _product(m, n, k, dtype, ldx, ldw, ldo)
    torch.cuda.empty_cache()


def test_product_repeats_its_bits():
    say("product repeats")
    r = np.random.default_rng(1)
    for m in (8, 1700):
        x, _ = _rand8(r, m, 1024)
        w, _ = _rand8(r, 4096, 1024)
        xs = torch.rand((m, 8), device=DEV)
        ws = torch.rand((32, 8), device=DEV)
        outs = [torch.empty((m, 4096), device=DEV) for _ in range(3)]
        for o in outs:
            M.moe_gemm_fp8(x, 1024, xs, w, 1024, ws, m, 4096, 1024, o, M.MOE_DTYPE_F32, 4096)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ------------------------------------------------------------ routed experts

def _blobs(r, E, H, I):
    """Device blobs by the library's quantiser, and their values."""
    off, total = M.moe_fp8_blob_layout(H, I)
    dev = torch.full((E, total), 0x7F, dtype=torch.uint8, device=DEV)
    vals = []
    for e in range(E):
        each = []
        for j, (n, c) in enumerate(((I, H), (I, H), (H, I))):
            w = torch.from_numpy((r.normal(0, 0.02, (n, c)) * np.exp(r.normal(0, 1))).astype(
                np.float32)).to(DEV)
            ns = R.blocks(n) * R.blocks(c)
            q = dev[e, off[j]:off[j] + n * c]
            s = torch.empty(ns, device=DEV)
            M.moe_quantize_fp8(w, M.MOE_DTYPE_F32, c, n, c, 128, 0, q, c, s)
            dev[e, off[3 + j]:off[3 + j] + 4 * ns] = s.view(torch.uint8)
            each.append((R.codes(q).reshape(n, c), s.cpu().numpy().reshape(R.blocks(n), -1)))
        vals.append(each)
    table = dev.data_ptr() + total * torch.arange(E, dtype=torch.int64)
    return dev, vals, table.to(DEV)


def _grouping(idx, E):
    """Device perm, offsets of host idx [T, k] by moe_permute (ids outside
    0..E-1 are left out)."""
    T, k = idx.shape
    d = torch.from_numpy(np.ascontiguousarray(idx, np.int32)).to(DEV)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)   # noqa: E731
    counts, offsets, perm, inv = i32(E), i32(E + 1), i32(T * k), i32(T * k)
    n = M.moe_permute_workspace_bytes(T, k, E)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    M.moe_permute(d, T, k, E, counts, offsets, perm, inv, ws, n)
    return perm, offsets


def _ffn(x, perm, offsets, table, T, H, I, E, k, regime=M.MOE_REGIME_AUTO):
    r, n = M.moe_expert_ffn_w8a8_plan(T, H, I, E, k, regime)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device=DEV)
    y = torch.full((T * k + 2, H), -7.0, dtype=torch.float16, device=DEV)
    M.moe_expert_ffn_w8a8(x, perm, offsets, table, T, H, I, E, k, r, y, ws, n)
    torch.cuda.synchronize()
    return y


def _check_ffn(y, x, perm, offsets, vals, k, skip=()):
    perm, offsets = perm.cpu().numpy(), offsets.cpu().numpy()
    x = x.float().cpu().numpy()
    y = y.double().cpu().numpy()
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        if e in skip:
            assert (y[a:b] == -7.0).all()
            continue
        ref, bound = R.experts_row(x[perm[a:b] // k], *vals[e])
        tol = bound + 2.0 ** -11 * (np.abs(ref) + bound) + 2.0 ** -25
        off = np.abs(y[a:b] - ref) - tol
        assert np.all(off <= 0), "expert %d: %g over the bound" % (e, off.max())
    assert (y[int(offsets[-1]):] == -7.0).all()


FFN = [   # T, H, I, E, k, regime
    (1, 256, 512, 8, 2, 0), (1, 2048, 1024, 16, 8, 0), (4, 256, 192, 8, 2, 0),
    (3, 320, 64, 5, 3, 0), (1, 64, 64, 1, 1, 0), (4, 256, 192, 8, 2, M.MOE_REGIME_BATCHED),
    (5, 256, 192, 8, 2, 0), (16, 320, 64, 5, 3, M.MOE_REGIME_DECODE), (16, 320, 64, 5, 3, 0),
    (11, 2048, 1408, 6, 2, 0), (1, 8192, 64, 2, 1, 0), (9, 64, 8192, 2, 2, 0),
    (10, 64, 8192, 2, 2, 0), (40, 512, 320, 8, 4, 0),
    (17, 320, 64, 5, 3, M.MOE_REGIME_BATCHED), (40, 512, 320, 8, 4, M.MOE_REGIME_BATCHED),
    (128, 256, 192, 8, 1, M.MOE_REGIME_DECODE), (100, 2048, 512, 3, 1, M.MOE_REGIME_DECODE),
    (33, 4096, 128, 2, 2, M.MOE_REGIME_DECODE), (100, 256, 192, 4, 2, 0), (300, 512, 448, 3, 1, 0), (70, 2048, 512, 70, 4, 0)]


@pytest.mark.parametrize("T,H,I,E,k,regime", FFN)
def test_experts(T, H, I, E, k, regime):
    say("experts T=%d H=%d I=%d E=%d k=%d regime=%d" % (T, H, I, E, k, regime))
    r = np.random.default_rng(T * 17 + H + I)
    dev, vals, table = _blobs(r, E, H, I)
    x = torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV)
    idx = np.argsort(r.normal(0, 1, (T, E)) + np.linspace(0, 3, E), 1)[:, :k]
    perm, offsets = _grouping(idx, E)
    y = _ffn(x, perm, offsets, table, T, H, I, E, k, regime)
    _check_ffn(y, x, perm, offsets, vals, k)


@pytest.mark.parametrize("T", [2, 4, 16, 30, 60])
def test_experts_uneven(T):
    """Every token with the same expert twice, ids that route nowhere (rows
    behind the last sorted row stay as they were), and an absent expert."""
    say("experts uneven T=%d" % T)
    H, I, E, k = 256, 128, 6, 5
    r = np.random.default_rng(T)
    dev, vals, table = _blobs(r, E, H, I)
    x = torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV)
    x[0] = 0.0                                                # a token of zeros
    idx = np.tile(np.array([3, 3, -1, 5, 1]), (T, 1))
    idx[-1] = [4, 4, 4, 4, 4]
    perm, offsets = _grouping(idx, E)
    table[5] = 0
    y = _ffn(x, perm, offsets, table, T, H, I, E, k)
    _check_ffn(y, x, perm, offsets, vals, k, skip=(5,))


def test_experts_short_tiles():
    """Tiles of 192 rows whose last one holds one, two or three row fragments
    of each wave, or none of some; ragged fragments; an expert of one row."""
    say("experts short tiles")
    H, I, k = 192, 4096, 1
    rows = [193, 300, 129, 1, 64, 192, 241]
    E, T = len(rows), sum(rows)
    r = np.random.default_rng(5)
    dev, vals, table = _blobs(r, E, H, I)
    x = torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV)
    idx = np.repeat(np.arange(E), rows)
    r.shuffle(idx)
    perm, offsets = _grouping(idx.reshape(T, 1), E)
    y = _ffn(x, perm, offsets, table, T, H, I, E, k)
    _check_ffn(y, x, perm, offsets, vals, k)


@pytest.mark.parametrize("T", [3, 40, 120])
def test_experts_non_finite_tokens(T):
    """A token with a NaN or an infinity has rows without a finite value; every
    other row keeps its bits."""
    say("experts non-finite T=%d" % T)
    H, I, E, k = 256, 192, 5, 2
    r = np.random.default_rng(T)
    dev, vals, table = _blobs(r, E, H, I)
    x = torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV)
    perm, offsets = _grouping(np.argsort(r.normal(0, 1, (T, E)), 1)[:, :k], E)
    clean = _ffn(x, perm, offsets, table, T, H, I, E, k)
    for v in (float("nan"), float("inf"), -float("inf")):
        bad = x.clone()
        bad[1, 70] = v
        y = _ffn(bad, perm, offsets, table, T, H, I, E, k)
        hit = torch.cat([perm // k == 1, torch.zeros(2, dtype=torch.bool, device=DEV)])
        assert not bool(torch.isfinite(y[hit]).any())
        assert torch.equal(y[~hit], clean[~hit])


def test_experts_no_rows():
    """Nothing routed: nothing written."""
    say("experts no rows")
    H, I, E, k = 256, 128, 6, 2
    dev, vals, table = _blobs(np.random.default_rng(0), E, H, I)
    for T in (2, 20, 120):
        x = torch.ones((T, H), dtype=torch.float16, device=DEV)
        perm, offsets = _grouping(np.full((T, k), -1), E)
        assert bool((_ffn(x, perm, offsets, table, T, H, I, E, k) == -7.0).all())


@pytest.mark.parametrize("T", [1, 48, 150])
def test_experts_on_another_stream_and_captured(T):
    """A side stream gives the same bits; a captured call follows its buffers
    over replays, with eager calls on another workspace between them."""
    say("experts stream and graph T=%d" % T)
    H, I, E, k = 512, 256, 8, 2
    r = np.random.default_rng(T)
    dev, vals, table = _blobs(r, E, H, I)
    xs = [torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV) for _ in range(3)]
    idx = np.argsort(r.normal(0, 1, (T, E)), 1)[:, :k]
    perm, offsets = _grouping(idx, E)
    eager = [_ffn(x, perm, offsets, table, T, H, I, E, k) for x in xs]
    reg, n = M.moe_expert_ffn_w8a8_plan(T, H, I, E, k)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    y = torch.full_like(eager[0], -7.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.moe_expert_ffn_w8a8(xs[0], perm, offsets, table, T, H, I, E, k, reg, y, ws, n, side)
    side.synchronize()
    assert torch.equal(y, eager[0])
    xb = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_expert_ffn_w8a8(xb, perm, offsets, table, T, H, I, E, k, reg, y, ws, n)
    for i in (1, 2, 0):
        xb.copy_(xs[i])
        g.replay()
        again = _ffn(xs[i], perm, offsets, table, T, H, I, E, k)
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i]) and torch.equal(again, eager[i])
