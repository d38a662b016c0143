"""Norms without weights in a stack.  The library's calls are recorded, not made; no
GPU is touched."""
import pytest
import torch

import int4_weight_only_router_amd as M
from int4_weight_only_router_amd import layer as L
from int4_weight_only_router_amd.layer import BlockNorms, MoELayer, block_norm

H = 256
F16, F32 = M.MOE_DTYPE_F16, M.MOE_DTYPE_F32


def w(dtype=torch.float16):
    return torch.ones(H, dtype=dtype)


def _layer(norms):
    return MoELayer(H, 64, 4, 2, 64, torch.zeros((4, H), dtype=torch.float16),
                    torch.zeros(4, dtype=torch.int64), device="cpu", norms=norms)


@pytest.fixture
def calls(monkeypatch):
    """Arguments of the library's calls, in order; none of them runs."""
    made = []
    monkeypatch.setattr(L.A, "moe_block_norm", lambda *a, **k: made.append(a))
    for name in ("route_permute", "experts", "combine"):
        monkeypatch.setattr(MoELayer, name, lambda *a, **k: None)
    return made


def _types(calls):
    return [a[12] for a in calls]


PLAIN, POST = BlockNorms(), BlockNorms(post=True, scale=0.5)
W16, W32 = BlockNorms(w()), BlockNorms(w(torch.float32))
P32 = BlockNorms(None, post=True, post_w=w(torch.float32))


@pytest.mark.parametrize("norms,types", [
    ((PLAIN, W32), [F16, F32, None]), ((W32, PLAIN), [F32, None, None]),
    ((POST, W32, PLAIN), [None, F32, None, None]), ((PLAIN, W16, POST), [None, F16, None, None]),
    ((P32, PLAIN), [None, F32, None]), ((PLAIN, P32), [None, None, F32]),
    ((PLAIN, P32, W32), [None, None, F32, None]), ((PLAIN, POST), [None, None, None])])
def test_stack_of_norms_without_weights(calls, norms, types):
    """A layer without weights stands next to weights of either type; the call says
    the type of those that there are."""
    layers = [_layer(n) for n in norms]
    acts = [torch.zeros((1, H), dtype=torch.float16) for _ in range(len(layers) + 1)]
    L.stack_forward(layers, [lay.buffers(1) for lay in layers], acts)
    got = _types(calls)
    assert len(got) == len(types)
    for g, t, a in zip(got, types, calls):
        given = [v for v in (a[7], a[8], a[9], a[10]) if v is not None]
        if given:
            assert g == (F32 if given[0].dtype == torch.float32 else F16)
        assert t is None or g == t


@pytest.mark.parametrize("norms", [(W16, PLAIN, W32), (P32, W16), (W16, P32)])
def test_stack_refuses_weights_of_two_types(calls, norms):
    layers = [_layer(n) for n in norms]
    acts = [torch.zeros((1, H), dtype=torch.float16) for _ in range(len(layers) + 1)]
    with pytest.raises(ValueError, match="one type"):
        L.stack_forward(layers, [lay.buffers(1) for lay in layers], acts)
    assert not calls


def test_one_call_of_two_types(calls):
    h = torch.zeros((1, H), dtype=torch.float16)
    with pytest.raises(ValueError, match="one type"):
        block_norm(h, h, P32, W16, h, h)
    block_norm(h, h, P32, PLAIN, h, h)
    block_norm(h, h, BlockNorms(w(), post=True), W32, h, h)   # (its pre weights belong elsewhere)
    assert _types(calls) == [F32, F32]
