"""MoELayer.balance and router_backward refuse buffers and tensors that their kernels
would read or write past the end of.  The library's calls are recorded, not made; no
GPU is touched."""
import pytest
import torch

from int4_weight_only_router_amd import layer as L
from int4_weight_only_router_amd.layer import MoELayer

H = 256


def _layer(E=4, H=H):
    return MoELayer(H, 64, E, 2, 64, torch.zeros((E, H), dtype=torch.float16),
                    torch.zeros(E, dtype=torch.int64), device="cpu")


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in ("moe_balance_loss", "moe_linear_f16_backward", "moe_router_logits"):
        monkeypatch.setattr(L.A, name, lambda *a, _n=name, **k: made.append(_n))
    return made


def test_balance_takes_its_own_buffers_only(calls):
    """Buffers of other experts or widths, and rows of other counts, are not written or
    read past their end."""
    lay = _layer()
    x, b, g = torch.zeros((3, H), dtype=torch.float16), lay.buffers(3), lay.balance_buffers(3)
    up = torch.ones(1)
    for other in (_layer(E=3), _layer(H=512), _layer(E=8, H=2048)):
        with pytest.raises(ValueError, match="buffers"):
            lay.balance(x, b, other.balance_buffers(3), 0.1, d_loss=up)
    for bad in (x[:2], torch.zeros((4, H), dtype=torch.float16), torch.zeros((3, H - 8), dtype=torch.float16)):
        with pytest.raises(ValueError, match="rows"):
            lay.balance(bad, b, g, 0.1, d_loss=up)
    for kw in (dict(d_loss=torch.ones(1, device="meta")),
               dict(mask=torch.ones(3, dtype=torch.uint8, device="meta"))):
        with pytest.raises(ValueError, match="device"):
            lay.balance(x, b, g, 0.1, **kw)
    assert not calls
    lay.balance(x, b, g, 0.1, d_loss=up)
    for bad in (x[:2], torch.zeros((3, H + 8), dtype=torch.float16)):
        with pytest.raises(ValueError, match="rows"):
            lay.router_backward(bad, g)
    with pytest.raises(ValueError, match="buffers"):
        _layer(E=3).router_backward(x, g)
    assert calls == ["moe_router_logits", "moe_balance_loss"]
    lay.router_backward(x, g)
    assert calls[-1] == "moe_linear_f16_backward"
