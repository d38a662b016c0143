"""What moe_linear_f16_backward answers on the host about dz's precision."""
import pytest

import int4_weight_only_router_amd as M

P = 4096
F16, F32, DZ = M.MOE_DTYPE_F16, M.MOE_DTYPE_F32, M.MOE_DZ_F16


def _code(m, n, k, act, dtype):
    with pytest.raises(M.MoEError) as ei:
        M.moe_linear_f16_backward(P, n, P, n, act, P, k, P, k, m, n, k, P, k, P, k, dtype, None,
                                  None, 0, stream=0)
    return ei.value.code


def test_flag():
    for act in range(5):
        assert _code(64, 64, 64, act, F16 | DZ) == M.MOE_ENOMEM   # (no workspace: taken)
    assert _code(64, 64, 64, M.MOE_ACT_NONE, F32 | DZ) == M.MOE_ENOMEM
    assert _code(64, 64, 64, M.MOE_ACT_SILU, F32 | DZ) == M.MOE_EUNSUPPORTED
    for bad in (2 | DZ, M.MOE_DTYPE_BF16 | DZ, F16 | M.MOE_ACC_F32, F16 | DZ << 1):
        assert _code(64, 64, 64, M.MOE_ACT_NONE, bad) == M.MOE_EINVAL
    with pytest.raises(M.MoEError) as ei:   # no flag of the forward call
        M.moe_linear_f16(P, 64, P, 64, None, 0, None, 0, 4, 32, 64, P, F16 | DZ, 32, stream=0)
    assert ei.value.code == M.MOE_EINVAL


@pytest.mark.parametrize("act", [M.MOE_ACT_SILU, M.MOE_ACT_GELU, M.MOE_ACT_GELU_TANH])
def test_rows_of_a_dz_of_two(act):
    """k of dw is passed twice: half as many rows, or dz rounded."""
    m = 1 << 29
    assert _code(m, 8, 8, act, F16) == M.MOE_ENOMEM
    assert _code(m + 1, 8, 8, act, F16) == M.MOE_EUNSUPPORTED
    assert _code(m + 1, 8, 8, act, F16 | DZ) == M.MOE_ENOMEM
    for free in (M.MOE_ACT_NONE, M.MOE_ACT_RELU):
        assert _code(m + 1, 8, 8, free, F16) == M.MOE_ENOMEM
    assert _code(2, 1 << 22, 8, act, F16) == M.MOE_ENOMEM
