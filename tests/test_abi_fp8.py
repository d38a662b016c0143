"""Refusals of the score-routing and FP8 entry points: everything below fails
on the host, before anything is launched; no GPU is touched."""
import pytest

import int4_weight_only_router_amd as M

EINVAL, EUNSUP, ENOMEM = M.MOE_EINVAL, M.MOE_EUNSUPPORTED, M.MOE_ENOMEM
F32, F16, BF16 = M.MOE_DTYPE_F32, M.MOE_DTYPE_F16, M.MOE_DTYPE_BF16
P = 4096   # an aligned address that no call below reads


def _code(f, *args, **kw):
    with pytest.raises(M.MoEError) as ei:
        f(*args, **kw)
    assert M.moe_last_error()
    return ei.value.code


def _select(logits=P, dtype=F32, ld=64, bias=None, T=2, E=64, k=8, score=0, n=4, keep=2, flags=0,
            scale=1.0, idx=P, w=P):
    return (logits, dtype, ld, bias, T, E, k, score, n, keep, flags, scale, idx, w)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(E=0), EINVAL), (dict(k=0), EINVAL), (dict(k=65), EINVAL),
    (dict(dtype=M.MOE_DTYPE_F32_PM), EINVAL), (dict(dtype=9), EINVAL), (dict(score=2), EINVAL),
    (dict(flags=4), EINVAL), (dict(n=0), EINVAL), (dict(n=3), EINVAL), (dict(keep=0), EINVAL),
    (dict(keep=5), EINVAL), (dict(n=16, keep=1), EINVAL), (dict(ld=63), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(logits=None), EINVAL), (dict(idx=None), EINVAL), (dict(w=None), EINVAL),
    (dict(logits=P + 2), EINVAL), (dict(logits=P + 1, dtype=F16), EINVAL),
    (dict(bias=P + 2), EINVAL), (dict(idx=P + 2), EINVAL), (dict(w=P + 1), EINVAL),
    (dict(T=(1 << 25) + 1), EUNSUP),
    (dict(E=2048, ld=2048), EUNSUP), (dict(k=17, n=1, keep=1), EUNSUP),
    (dict(E=130, ld=130, n=65, keep=65), EUNSUP)])
def test_select_refusals(kw, code):
    args = _select(**kw)
    assert _code(M.moe_route_select, *args, stream=0) == code
    assert _code(M.moe_route_select_permute, *args, P, P, P, P, P, 1 << 30, stream=0) == code


def test_select_permute_refusals():
    assert _code(M.moe_route_select_permute, *_select(), None, P, P, P, P, 1 << 20,
                 stream=0) == EINVAL
    big = _select(T=100000)
    need = M.moe_route_select_workspace_bytes(100000, 8, 64)
    assert need > 0
    assert _code(M.moe_route_select_permute, *big, P, P, P, P, P, need - 1, stream=0) == ENOMEM
    assert _code(M.moe_route_select_permute, *big, P, P, P, P, None, need, stream=0) == ENOMEM
    assert _code(M.moe_route_select_permute, *big, P, P, P, P, P + 8, need, stream=0) == EINVAL
    assert _code(M.moe_route_select_permute, *big, P, P, P + 2, P, P, need, stream=0) == EINVAL
    assert M.moe_route_select_workspace_bytes(1, 8, 64) == 0
    M.moe_route_select(*_select(T=0, logits=None, idx=None, w=None), stream=0)   # no-op


@pytest.mark.parametrize("args,code", [
    ((P, P, None, -1, 2048, 64, P), EINVAL), ((P, P, None, 1, 2044, 64, P), EINVAL),
    ((P, P, None, 1, 768, 64, P), EUNSUP), ((P, P, None, 1, 2048, 1025, P), EUNSUP),
    ((None, P, None, 1, 2048, 64, P), EINVAL), ((P, P, None, 1, 2048, 64, None), EINVAL),
    ((P + 8, P, None, 1, 2048, 64, P), EINVAL)])
def test_logits_refusals(args, code):
    assert _code(M.moe_router_logits, *args, stream=0) == code


def _quant(x=P, dtype=F16, ldx=256, rows=3, cols=256, block=1, flags=0, q=P, ldq=256, s=P):
    return (x, dtype, ldx, rows, cols, block, flags, q, ldq, s)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=0), EINVAL),
    (dict(ldx=255), EINVAL), (dict(ldq=255), EINVAL), (dict(block=64), EINVAL),
    (dict(flags=2), EINVAL), (dict(x=None), EINVAL), (dict(q=None), EINVAL), (dict(s=None), EINVAL),
    (dict(x=P + 1), EINVAL), (dict(s=P + 2), EINVAL), (dict(rows=1 << 40), EUNSUP),
    (dict(cols=(1 << 30) + 1, ldx=1 << 31, ldq=1 << 31), EUNSUP)])
def test_quantize_refusals(kw, code):
    assert _code(M.moe_quantize_fp8, *_quant(**kw), stream=0) == code


def test_quantize_no_rows():
    M.moe_quantize_fp8(*_quant(rows=0, x=None, q=None, s=None), stream=0)


def _gemm(xq=P, ldx=256, xs=P, wq=P, ldw=256, ws=P, m=4, n=64, k=256, out=P, dt=F16, ldo=64):
    return (xq, ldx, xs, wq, ldw, ws, m, n, k, out, dt, ldo)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), EINVAL), (dict(m=-1), EINVAL), (dict(n=0), EINVAL), (dict(k=0), EINVAL),
    (dict(ldx=240), EINVAL), (dict(ldw=240), EINVAL), (dict(ldo=63), EINVAL),
    (dict(k=250), EUNSUP), (dict(ldx=264), EUNSUP), (dict(ldw=264), EUNSUP),
    (dict(k=16400, ldx=16400, ldw=16400), EUNSUP), (dict(xq=None), EINVAL), (dict(xs=None), EINVAL),
    (dict(wq=None), EINVAL), (dict(ws=None), EINVAL), (dict(out=None), EINVAL),
    (dict(xq=P + 8), EINVAL), (dict(wq=P + 4), EINVAL), (dict(xs=P + 2), EINVAL),
    (dict(out=P + 1), EINVAL), (dict(out=P + 2, dt=F32), EINVAL),
    (dict(m=2097121, ldw=1 << 22), EUNSUP), (dict(m=0x7fffff01), EUNSUP),
    (dict(n=0x7fffff01, ldo=1 << 31), EUNSUP),
    (dict(n=(1 << 28) + 1, ldo=1 << 31, ldw=1 << 22), EUNSUP),
    (dict(m=1 << 24, n=1 << 24, ldo=1 << 24), EUNSUP)])
def test_product_refusals(kw, code):
    assert _code(M.moe_gemm_fp8, *_gemm(**kw), stream=0) == code


def test_product_no_rows():
    M.moe_gemm_fp8(*_gemm(m=0, xq=None, out=None), stream=0)


@pytest.mark.parametrize("args,code", [
    ((-1, 2048, 1024, 64, 8), EINVAL), ((1, 0, 1024, 64, 8), EINVAL), ((1, 2048, 1024, 4, 5), EINVAL),
    ((1, 2080, 1024, 64, 8), EUNSUP), ((1, 2048, 1000, 64, 8), EUNSUP),
    ((1, 8256, 1024, 64, 8), EUNSUP), ((1, 2048, 1024, 2048, 8), EUNSUP),
    ((1, 2048, 1024, 64, 17), EUNSUP), ((1, 2048, 1024, 64, 8, M.MOE_REGIME_SMALL), EINVAL),
    ((1, 2048, 1024, 64, 8, M.MOE_REGIME_AUTO | M.MOE_Y_TOKEN_ORDER), EINVAL),
    ((129, 2048, 1024, 64, 8, M.MOE_REGIME_DECODE), EUNSUP),
    ((10, 64, 8192, 64, 8, M.MOE_REGIME_DECODE), EUNSUP)])
def test_plan_refusals(args, code):
    assert _code(M.moe_expert_ffn_w8a8_plan, *args) == code


def test_plan_and_layout():
    assert M.moe_expert_ffn_w8a8_plan(4, 2048, 1024, 64, 8)[0] == M.MOE_REGIME_DECODE
    assert M.moe_expert_ffn_w8a8_plan(8, 2048, 1024, 64, 8)[0] == M.MOE_REGIME_DECODE
    assert M.moe_expert_ffn_w8a8_plan(9, 2048, 1024, 64, 8)[0] == M.MOE_REGIME_BATCHED
    assert M.moe_expert_ffn_w8a8_plan(16, 2048, 1024, 8, 2)[0] == M.MOE_REGIME_DECODE
    assert M.moe_expert_ffn_w8a8_plan(64, 2048, 1024, 8, 1)[0] == M.MOE_REGIME_DECODE
    assert M.moe_expert_ffn_w8a8_plan(65, 2048, 1024, 8, 1)[0] == M.MOE_REGIME_BATCHED
    assert M.moe_expert_ffn_w8a8_plan(96, 640, 1024, 8, 2)[0] == M.MOE_REGIME_DECODE
    assert M.moe_expert_ffn_w8a8_plan(97, 256, 1024, 8, 2)[0] == M.MOE_REGIME_BATCHED
    assert M.moe_expert_ffn_w8a8_plan(86, 768, 1024, 8, 2)[0] == M.MOE_REGIME_BATCHED
    assert M.moe_expert_ffn_w8a8_plan(129, 256, 1024, 8, 1)[0] == M.MOE_REGIME_BATCHED
    assert M.moe_expert_ffn_w8a8_plan(9, 64, 8192, 8, 2)[0] == M.MOE_REGIME_DECODE
    assert M.moe_expert_ffn_w8a8_plan(10, 64, 8192, 8, 2)[0] == M.MOE_REGIME_BATCHED
    r, n = M.moe_expert_ffn_w8a8_plan(4096, 2048, 1024, 64, 8)
    assert r == M.MOE_REGIME_BATCHED and n >= 4096 * (2048 + 8 * 1024)
    off, total = M.moe_fp8_blob_layout(320, 192)
    assert off == [0, 61440, 122880, 184320, 184576, 184832] and total == 185088
    assert _code(M.moe_fp8_blob_layout, 0, 64) == EINVAL


def test_experts_refusals():
    a = (P, P, P, P, 8, 256, 128, 8, 2, M.MOE_REGIME_BATCHED, P, P)
    need = M.moe_expert_ffn_w8a8_plan(8, 256, 128, 8, 2, M.MOE_REGIME_BATCHED)[1]
    assert _code(M.moe_expert_ffn_w8a8, *a, need - 1, stream=0) == ENOMEM
    for i in (0, 1, 2, 3, 10):
        b = list(a)
        b[i] = None
        assert _code(M.moe_expert_ffn_w8a8, *b, need, stream=0) == EINVAL
    for i in (0, 10, 11):
        b = list(a)
        b[i] = P + 8
        assert _code(M.moe_expert_ffn_w8a8, *b, need, stream=0) == EINVAL
    b = list(a)
    b[11] = None
    assert _code(M.moe_expert_ffn_w8a8, *b, need, stream=0) == ENOMEM
    M.moe_expert_ffn_w8a8(None, None, None, None, 0, 256, 128, 8, 2, M.MOE_REGIME_BATCHED, None,
                          None, 0, stream=0)   # no tokens
