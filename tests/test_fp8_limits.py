"""Size limits of the FP8 and score-routing entry points that are answered on
the host, before any of a call's launches; no GPU is touched."""
import pytest

import int4_weight_only_router_amd as M

P = 4096   # an aligned address that no call below reads


def _unsupported(f, *args, **kw):
    with pytest.raises(M.MoEError) as ei:
        f(*args, **kw)
    assert ei.value.code == M.MOE_EUNSUPPORTED


@pytest.mark.parametrize("T,H,I,E,k", [
    (1 << 21, 64, 8192, 16, 16),             # gate/up: too many tiles of h
    (1 << 23, 8192, 128, 8, 8),              # down: too many tiles of y
    ((1 << 22) + 1, 8192, 64, 1, 1),         # too many token blocks to quantise
])
@pytest.mark.parametrize("regime", [M.MOE_REGIME_AUTO, M.MOE_REGIME_BATCHED])
def test_experts_beyond_a_launch(T, H, I, E, k, regime):
    """Refused by the plan and so by the call, which asks it first."""
    _unsupported(M.moe_expert_ffn_w8a8_plan, T, H, I, E, k, regime)
    _unsupported(M.moe_expert_ffn_w8a8, P, P, P, P, T, H, I, E, k, regime, P, P, 1 << 60, stream=0)


def test_experts_at_the_limits():
    # (16 T / 192 + 16) * 64 tiles of h just fit; another row tile does not
    T = (((1 << 23) - 8) // 64 - 16) * 192 // 16
    assert M.moe_expert_ffn_w8a8_plan(T, 64, 8192, 16, 16)[0] == M.MOE_REGIME_BATCHED
    _unsupported(M.moe_expert_ffn_w8a8_plan, T + 12, 64, 8192, 16, 16)
    assert M.moe_expert_ffn_w8a8_plan((1 << 28) - 32, 64, 64, 8, 1)[0] == M.MOE_REGIME_BATCHED
    _unsupported(M.moe_expert_ffn_w8a8_plan, (1 << 28) - 31, 64, 64, 8, 1)


def test_blob_layout_beyond_64_bits():
    off, total = M.moe_fp8_blob_layout(1 << 30, 1 << 30)
    assert off[:4] == [0, 1 << 60, 2 << 60, 3 << 60]
    assert off[4] - off[3] == 4 << 46 and total == off[5] + (4 << 46)
    for H, I in (((1 << 30) + 1, 64), (64, (1 << 31) - 1), ((1 << 31) - 1, (1 << 31) - 1)):
        _unsupported(M.moe_fp8_blob_layout, H, I)


@pytest.mark.parametrize("T", [(1 << 27) - 7, (1 << 31) - 1])
def test_logits_beyond_a_launch(T):
    _unsupported(M.moe_router_logits, P, P, None, T, 256, 64, P, stream=0)


def test_fp32_sums_flag():
    """The plan keeps the flag in what it resolves, and asks for the same workspace."""
    for T, regime in ((1, M.MOE_REGIME_AUTO), (1, M.MOE_REGIME_BATCHED), (500, M.MOE_REGIME_AUTO)):
        r, n = M.moe_expert_ffn_w8a8_plan(T, 256, 128, 8, 2, regime)
        assert M.moe_expert_ffn_w8a8_plan(T, 256, 128, 8, 2, regime | M.MOE_ACC_F32) == \
            (r | M.MOE_ACC_F32, n)
    for call in (lambda: M.moe_expert_ffn_w8a8_plan(1, 256, 128, 8, 2, M.MOE_REGIME_SMALL | M.MOE_ACC_F32),
                 lambda: M.moe_gemm_fp8(P, 256, P, P, 256, P, 4, 64, 256, P, 2 | M.MOE_ACC_F32, 64,
                                        stream=0),
                 lambda: M.moe_expert_ffn_plan(1, 256, 128, 8, 2, 64, M.MOE_ACC_F32)):
        with pytest.raises(M.MoEError) as ei:
            call()
        assert ei.value.code == M.MOE_EINVAL
