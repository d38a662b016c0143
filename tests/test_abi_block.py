"""Refusals of the operators around a routed block: everything below fails on the
host, before anything is launched; no GPU is touched."""
import pytest

import int4_weight_only_router_amd as M

EINVAL, EUNSUP, ENOMEM = M.MOE_EINVAL, M.MOE_EUNSUPPORTED, M.MOE_ENOMEM
F32, F16, BF16 = M.MOE_DTYPE_F32, M.MOE_DTYPE_F16, M.MOE_DTYPE_BF16
P = 4096   # an aligned address that no call below reads
NAN, INF = float("nan"), float("inf")


def _code(f, *args, **kw):
    with pytest.raises(M.MoEError) as ei:
        f(*args, **kw)
    assert M.moe_last_error()
    return ei.value.code


def _norm(y=P, ldy=64, r=P, ldr=64, gate=P, ldg=0, scale=1.0, pw=P, pb=P, qw=P, qb=P, dt=F16,
          wt=F16, kind=0, flags=1, eps=1e-5, T=2, H=64, out=P, ldo=64, n=P, ldn=64):
    return (y, ldy, r, ldr, gate, ldg, scale, pw, pb, qw, qb, dt, wt, kind, flags, eps, T, H, out,
            ldo, n, ldn)


NORM = [
    (dict(dt=2), EINVAL), (dict(dt=9), EINVAL), (dict(wt=BF16), EINVAL), (dict(dt=F32), EINVAL),
    (dict(kind=2), EINVAL), (dict(flags=5), EINVAL), (dict(T=-1), EINVAL), (dict(H=0), EINVAL),
    (dict(eps=-1e-6), EINVAL), (dict(eps=NAN), EINVAL), (dict(eps=INF), EINVAL),
    (dict(scale=INF), EINVAL), (dict(scale=NAN), EINVAL), (dict(H=8193), EUNSUP),
    (dict(ldg=63), EINVAL), (dict(ldg=-64), EINVAL), (dict(gate=None, ldg=64), EINVAL),
    (dict(flags=0), EINVAL), (dict(flags=0, pw=None), EINVAL), (dict(pw=P + 1), EINVAL),
    (dict(wt=F32, pb=P + 2), EINVAL), (dict(ldy=63), EINVAL), (dict(ldr=63), EINVAL),
    (dict(y=P + 1), EINVAL), (dict(r=P + 1), EINVAL), (dict(gate=P + 1), EINVAL),
    (dict(dt=F32, wt=F32, r=P + 2), EINVAL), (dict(y=None), EINVAL),
    (dict(y=None, gate=None), EINVAL), (dict(y=None, r=None, gate=None), EINVAL)]


@pytest.mark.parametrize("kw,code", NORM + [
    (dict(ldo=63), EINVAL), (dict(ldn=63), EINVAL), (dict(out=P + 1), EINVAL),
    (dict(n=P + 1), EINVAL), (dict(out=None, n=None), EINVAL), (dict(n=None), EINVAL),
    (dict(qw=P + 1), EINVAL), (dict(qb=P + 1), EINVAL)])
def test_norm_refusals(kw, code):
    assert _code(M.moe_block_norm, *_norm(**kw), stream=0) == code


def test_norm_no_rows():
    M.moe_block_norm(*_norm(T=0, y=None, r=None, out=None, n=None), stream=0)


GRADS = dict(dy=P, dr=P, dg=P, dpw=P, dpb=P, dqw=P, dqb=P)


def _norm_backward(dout=P, dn=P, ws=P, ws_bytes=1 << 30, **kw):
    g = {k: kw.pop(k, v) for k, v in GRADS.items()}
    a = _norm(**kw)
    return (dout, a[19], dn, a[21]) + a[:9] + (a[9],) + a[11:18] + tuple(g.values()) + (ws, ws_bytes)


@pytest.mark.parametrize("kw,code", NORM + [
    (dict(ldo=63), EINVAL), (dict(ldn=63), EINVAL), (dict(dout=P + 1), EINVAL),
    (dict(dn=P + 1), EINVAL), (dict(dout=None, dn=None), EINVAL), (dict(dn=None), EINVAL),
    (dict(dn=None, qw=None, dqw=None), EINVAL), (dict(r=None), EINVAL),
    (dict(gate=None), EINVAL), (dict(dy=P + 1), EINVAL), (dict(dr=P + 1), EINVAL),
    (dict(dg=P + 2), EINVAL), (dict(dg=P + 1, ldg=64), EINVAL), (dict(dpw=P + 2), EINVAL),
    (dict(dqb=P + 1), EINVAL), (dict(pw=None, pb=None, flags=0), EINVAL),
    (dict(y=None, gate=None, pw=None, pb=None, flags=0, dpw=None, dpb=None, dg=None), EINVAL),
    (dict(ws=None), ENOMEM), (dict(ws_bytes=64), ENOMEM), (dict(ws=P + 8), EINVAL)])
def test_norm_backward_refusals(kw, code):
    assert _code(M.moe_block_norm_backward, *_norm_backward(**kw), stream=0) == code


def test_norm_workspace():
    assert M.moe_block_norm_backward_workspace_bytes(0, 64) == 0
    assert M.moe_block_norm_backward_workspace_bytes(1, 8192) >= 5 * 8192 * 4
    assert M.moe_block_norm_backward_workspace_bytes(1 << 30, 8192) < 1 << 27


def _linear(x=P, ldx=64, w=P, ldw=64, bias=P, act=0, res=P, ldr=32, m=4, n=32, k=64, out=P, dt=F16,
            ldo=32, z=P, ldz=32, ws=P, ws_bytes=1 << 40):
    return (x, ldx, w, ldw, bias, act, res, ldr, m, n, k, out, dt, ldo, z, ldz, ws, ws_bytes)


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), EINVAL), (dict(n=0), EINVAL), (dict(k=0), EINVAL), (dict(act=5), EINVAL),
    (dict(act=-1), EINVAL), (dict(dt=BF16), EINVAL), (dict(dt=2), EINVAL), (dict(ldx=56), EINVAL),
    (dict(ldw=56), EINVAL), (dict(ldo=31), EINVAL), (dict(ldr=31), EINVAL), (dict(ldz=31), EINVAL),
    (dict(k=60), EUNSUP), (dict(ldx=68), EUNSUP), (dict(ldw=68), EUNSUP), (dict(x=None), EINVAL),
    (dict(w=None), EINVAL), (dict(out=None), EINVAL), (dict(x=P + 8), EINVAL),
    (dict(w=P + 2), EINVAL), (dict(bias=P + 2), EINVAL), (dict(z=P + 1), EINVAL),
    (dict(out=P + 1), EINVAL), (dict(res=P + 1), EINVAL), (dict(dt=F32, out=P + 2), EINVAL)])
def test_linear_refusals(kw, code):
    assert _code(M.moe_linear_f16, *_linear(**kw), stream=0) == code


def test_linear_no_rows():
    M.moe_linear_f16(*_linear(m=0, x=None, out=None, res=None, z=None, ws=None, ws_bytes=0),
                     stream=0)
    assert M.moe_linear_f16_workspace_bytes(0, 64, 64) == 0


def _linear_backward(dy=P, lddy=32, z=P, ldz=32, act=2, x=P, ldx=64, w=P, ldw=64, m=4, n=32, k=64,
                     dx=P, lddx=64, dw=P, lddw=64, dt=F16, db=P, ws=P, ws_bytes=1 << 40):
    return (dy, lddy, z, ldz, act, x, ldx, w, ldw, m, n, k, dx, lddx, dw, lddw, dt, db, ws, ws_bytes)


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), EINVAL), (dict(n=0), EINVAL), (dict(k=0), EINVAL), (dict(act=7), EINVAL),
    (dict(dt=BF16), EINVAL), (dict(lddy=31), EINVAL), (dict(ldz=31), EINVAL), (dict(ldx=56), EINVAL),
    (dict(ldw=56), EINVAL), (dict(lddx=63), EINVAL), (dict(lddw=63), EINVAL), (dict(k=60), EUNSUP),
    (dict(ldx=68), EUNSUP), (dict(ldw=68), EUNSUP), (dict(dt=F32), EUNSUP),
    (dict(dx=None, dw=None, db=None), EINVAL), (dict(dy=None), EINVAL), (dict(z=None), EINVAL),
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(x=P + 8), EINVAL), (dict(w=P + 8), EINVAL),
    (dict(dy=P + 1), EINVAL), (dict(z=P + 1), EINVAL), (dict(db=P + 2), EINVAL),
    (dict(dx=P + 1), EINVAL), (dict(dw=P + 1), EINVAL), (dict(ws=None), ENOMEM),
    (dict(ws_bytes=16), ENOMEM), (dict(ws=P + 8), EINVAL)])
def test_linear_backward_refusals(kw, code):
    assert _code(M.moe_linear_f16_backward, *_linear_backward(**kw), stream=0) == code


@pytest.mark.parametrize("kw", [
    dict(ldx=(1 << 22) + 8), dict(ldw=(1 << 22) + 8), dict(m=(1 << 30) + 1), dict(n=(1 << 30) + 1, ldo=1 << 31,
                                                                              ldr=1 << 31, ldz=1 << 31),
    dict(m=1 << 29, n=1 << 20, ldo=1 << 20, ldr=1 << 20, ldz=1 << 20)])
def test_linear_limits(kw):
    assert _code(M.moe_linear_f16, *_linear(**kw), stream=0) == EUNSUP


@pytest.mark.parametrize("kw", [
    dict(ldx=(1 << 22) + 8), dict(ldw=(1 << 22) + 8), dict(m=(1 << 30) + 1),
    dict(m=(1 << 30) + 1, dx=None, dw=None), dict(m=(1 << 31) - 1, dx=None),
    dict(n=(1 << 22) + 1, lddy=1 << 23, ldz=1 << 23),
    dict(m=1 << 29, k=1 << 20, ldx=1 << 20, ldw=1 << 20, lddx=1 << 20, lddw=1 << 20, dx=None)])
def test_linear_backward_limits(kw):
    assert _code(M.moe_linear_f16_backward, *_linear_backward(**kw), stream=0) == EUNSUP
    a = dict(dict(m=4, n=32, k=64), **kw)
    if max(a.get("ldx", 0), a.get("ldw", 0), a["n"]) <= 1 << 22:   # (strides are not in the query)
        assert M.moe_linear_f16_backward_workspace_bytes(a["m"], a["n"], a["k"]) == 0


def _balance(l=P, dt=F32, ld=64, idx=P, mask=P, T=100, E=64, k=8, score=0, c=0.1, z=0.1, counts=P,
             mean=P, losses=P, up=P, dl=P, gt=F32, ldd=64, ws=P, ws_bytes=1 << 30):
    return (l, dt, ld, idx, mask, T, E, k, score, c, z, counts, mean, losses, up, dl, gt, ldd, ws,
            ws_bytes)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(E=0), EINVAL), (dict(k=0), EINVAL), (dict(k=65), EINVAL),
    (dict(dt=2), EINVAL), (dict(gt=2), EINVAL), (dict(score=2), EINVAL), (dict(c=INF), EINVAL),
    (dict(z=NAN), EINVAL), (dict(ld=63), EINVAL), (dict(ldd=63), EINVAL), (dict(l=None), EINVAL),
    (dict(counts=None), EINVAL), (dict(l=P + 2), EINVAL), (dict(l=P + 1, dt=F16), EINVAL),
    (dict(dl=P + 2), EINVAL), (dict(dl=P + 1, gt=BF16), EINVAL), (dict(idx=P + 2), EINVAL),
    (dict(counts=P + 1), EINVAL), (dict(mean=P + 2), EINVAL), (dict(losses=P + 2), EINVAL),
    (dict(up=P + 2), EINVAL), (dict(E=1025, ld=1025, ldd=1025), EUNSUP),
    (dict(T=1 << 28), EUNSUP), (dict(ws=None), ENOMEM), (dict(ws_bytes=64), ENOMEM),
    (dict(ws=P + 4), EINVAL)])
def test_balance_refusals(kw, code):
    assert _code(M.moe_balance_loss, *_balance(**kw), stream=0) == code


def test_balance_workspace():
    assert M.moe_balance_loss_workspace_bytes(0, 64) == 0
    assert M.moe_balance_loss_workspace_bytes(100, 1025) == 0
    assert 0 < M.moe_balance_loss_workspace_bytes(1 << 30, 1024) < 1 << 24
