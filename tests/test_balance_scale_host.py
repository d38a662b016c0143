"""Without a loss scale MoELayer.balance forms no gradient, and router_backward says so.
The library's calls are recorded, not made; no GPU is touched."""
import pytest
import torch

import int4_weight_only_router_amd as M
from int4_weight_only_router_amd import layer as L
from int4_weight_only_router_amd.layer import MoELayer


@pytest.mark.parametrize("scale", [1.0, 65536.0])
def test_gradient_needs_its_scale(monkeypatch, scale):
    made = []
    for name in ("moe_balance_loss", "moe_linear_f16_backward", "moe_router_logits"):
        monkeypatch.setattr(L.A, name, lambda *a, _n=name, **k: made.append((_n, a)))
    lay = MoELayer(256, 64, 4, 2, 64, torch.zeros((4, 256), dtype=torch.float16),
                   torch.zeros(4, dtype=torch.int64), device="cpu")
    x, b, g = torch.zeros((3, 256), dtype=torch.float16), lay.buffers(3), lay.balance_buffers(3)
    with pytest.raises(ValueError, match="d_loss"):   # nothing formed yet
        lay.router_backward(x, g)
    assert lay.balance(x, b, g, 0.1) is g.losses
    assert made[-1][1][15] is None   # dlogits
    with pytest.raises(ValueError, match="d_loss"):
        lay.router_backward(x, g)
    lay.balance(x, b, g, 0.1, d_loss=torch.full((1,), scale))
    assert made[-1][1][15] is g.dlogits and made[-1][1][16] == M.MOE_DTYPE_F16
    lay.router_backward(x, g)
    lay.balance(x, b, g, 0.1)   # the losses alone: what was formed is not this call's
    with pytest.raises(ValueError, match="d_loss"):
        lay.router_backward(x, g)
    assert [n for n, _ in made].count("moe_linear_f16_backward") == 1
