"""Limits of the operators around a routed block that are answered on the host, before
any launch: refused sizes by their code, sizes that are taken by the next refusal in
line (a null pointer).  No GPU is touched."""
import pytest

import int4_weight_only_router_amd as M

P = 4096   # an aligned address that no call below reads
F16, F32 = M.MOE_DTYPE_F16, M.MOE_DTYPE_F32


def _code(f, *args, **kw):
    with pytest.raises(M.MoEError) as ei:
        f(*args, **kw)
    return ei.value.code


def _forward(m, n, k):
    return _code(M.moe_linear_f16, None, k, P, k, None, 0, None, 0, m, n, k, P, F16, n, stream=0)


def _backward(m, n, k, act=0, dx=P, dw=P, db=P, dtype=F16, ws=None):
    return _code(M.moe_linear_f16_backward, P, n, P, n, act, P, k, P, k, m, n, k, dx, k, dw, k,
                 dtype, db, ws, 0, stream=0)


@pytest.mark.parametrize("m,n,k", [(1 << 28, 8, 8), (1 << 28, 64, 64), (1 << 29, 32, 64),
                                   (1 << 26, 1024, 8), (1 << 29, 128, 512)])
def test_products_that_some_tile_fits(m, n, k):
    """Narrow tall products: the fastest tiles would be more than a launch holds, wider
    ones are not."""
    assert _forward(m, n, k) == M.MOE_EINVAL   # (x is null)
    assert M.moe_linear_f16_workspace_bytes(m, n, k) == 0   # whole, not in parts


@pytest.mark.parametrize("m,n,k", [(1 << 30, 257, 64), (1 << 25, 8192, 64)])
def test_products_that_no_tile_fits(m, n, k):
    assert _forward(m, n, k) == M.MOE_EUNSUPPORTED


@pytest.mark.parametrize("outs", [dict(), dict(dx=None), dict(dw=None), dict(dx=None, dw=None)])
@pytest.mark.parametrize("m,n,k", [(1 << 28, 8, 8), (1 << 28, 64, 64)])
def test_gradients_that_some_tile_fits(m, n, k, outs):
    assert _backward(m, n, k, **outs) == M.MOE_ENOMEM   # (no workspace)
    assert M.moe_linear_f16_backward_workspace_bytes(m, n, k) > 0
