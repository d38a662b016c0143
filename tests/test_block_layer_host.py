"""What layers with norms refuse before any call into the library; no GPU is touched."""
import pytest
import torch

import int4_weight_only_router_amd as M
from int4_weight_only_router_amd.layer import BlockNorms, MoELayer, ScoreRouting, stack_forward

H = 256


def _layer(norms, H=H, routing=None, fmt=M.MOE_FMT_SYM):
    return MoELayer(H, 64, 4, 2, 64, torch.zeros((4, H), dtype=torch.float16),
                    torch.zeros(4, dtype=torch.int64), device="cpu", norms=norms, routing=routing,
                    fmt=fmt)


def _stack(*norms):
    layers = [_layer(n) for n in norms]
    bufs = [lay.buffers(1) for lay in layers]
    acts = [torch.zeros((1, H), dtype=torch.float16) for _ in range(len(layers) + 1)]
    return layers, bufs, acts


def w(dtype=torch.float16):
    return torch.ones(H, dtype=dtype)


@pytest.mark.parametrize("norms", [
    (BlockNorms(w()), None), (None, BlockNorms(w())),
    (BlockNorms(w()), BlockNorms(w(), eps=1e-6)),
    (BlockNorms(w()), BlockNorms(w(), kind=M.MOE_NORM_LAYER)),
    (BlockNorms(w()), BlockNorms(w(), unit_offset=True)),
    (BlockNorms(w()), BlockNorms(w(torch.float32)))])
def test_stack_refuses_mixed_norms(norms):
    with pytest.raises(ValueError, match="stack"):
        stack_forward(*_stack(*norms))


def test_norm_weights_of_one_type():
    with pytest.raises(ValueError, match="all be fp16 or all fp32"):
        BlockNorms(w(), post=True, post_w=w(torch.float32))
    with pytest.raises(ValueError, match="all be fp16 or all fp32"):
        BlockNorms(w(torch.bfloat16))
    assert BlockNorms(w(torch.float32)).w_dtype == M.MOE_DTYPE_F32
    assert BlockNorms().w_dtype == M.MOE_DTYPE_F16


def test_pool_takes_no_norms():
    lay = _layer(BlockNorms(w()))
    with pytest.raises(ValueError, match="norms"):
        lay.pool_args(lay.buffers(1), torch.zeros(2, dtype=torch.int32))


def test_buffers():
    """Only layers that need them hold a normed input and a workspace of the router."""
    b = _layer(BlockNorms(w())).buffers(3)
    assert b.normed.shape == (3, H) and b.router_ws is None
    assert _layer(None).buffers(3).normed is None
    wide = _layer(None, 2560, ScoreRouting(), M.MOE_FMT_FP8)
    assert not wide.pinned_router and wide.buffers(3).logits.shape == (3, 4)
    need = M.moe_linear_f16_workspace_bytes(3, 4, 2560)
    ws = wide.buffers(3).router_ws
    assert (0 if ws is None else ws.numel()) == need


@pytest.mark.parametrize("norms,match", [
    (BlockNorms(torch.ones(H - 1, dtype=torch.float16)), "values"),
    (BlockNorms(w(), gate=torch.ones(2 * H, dtype=torch.float16)), "values"),
    (BlockNorms(torch.ones(2 * H, dtype=torch.float16)[::2]), "contiguous"),
    (BlockNorms(w(), gate=w(torch.float32)), "gate"),
    (BlockNorms(w(), post_w=w()), "post")])
def test_layer_refuses_norms(norms, match):
    with pytest.raises(ValueError, match=match):
        _layer(norms)


def test_balance_refusals():
    lay = _layer(None)
    b, g = lay.buffers(3), lay.balance_buffers(3)
    x = torch.zeros((3, H), dtype=torch.float16)
    with pytest.raises(ValueError, match="tokens"):
        lay.balance(x, b, lay.balance_buffers(2), 0.1)
    for mask in (torch.ones(2, dtype=torch.uint8), torch.ones(3, dtype=torch.int32),
                 torch.ones(6, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="mask"):
            lay.balance(x, b, g, 0.1, mask=mask)
    with pytest.raises(ValueError, match="d_loss"):
        lay.balance(x, b, g, 0.1, d_loss=torch.ones(1, dtype=torch.float16))
    with pytest.raises(ValueError, match="rows"):
        lay.router_backward(x[:2], g)
