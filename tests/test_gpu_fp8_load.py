"""load_experts_fp8 on a stream of its own: ordered against the current stream
by events, without holding the host."""
import numpy as np
import pytest
import torch

from int4_weight_only_router_amd.layer import load_experts_fp8
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["object", "address", "default"])
def test_load_orders_streams_without_the_host(kind, monkeypatch):
    """The current stream is kept busy before the copies, and memory freed by
    the loader is written over at once: the blobs are those of a plain load."""
    say("fp8 load on another stream by %s" % kind)
    H, I = 1024, 512
    r = np.random.default_rng(4)
    w = [tuple(torch.from_numpy(r.normal(0, 0.02, s).astype(np.float32)).to(DEV).double()
               for s in ((I, H), (I, H), (H, I))) for _ in range(4)]
    want = load_experts_fp8(w, H, I, DEV)
    side = torch.cuda.Stream()
    stream = {"object": side, "address": side.cuda_stream, "default": 0}[kind]
    here = torch.cuda.Stream()
    torch.cuda.synchronize()
    with monkeypatch.context() as m, torch.cuda.stream(here):
        def held(*a, **k):
            raise AssertionError("the host waits")
        m.setattr(torch.cuda, "synchronize", held)
        big = torch.zeros(1 << 28, device=DEV)
        for _ in range(20):
            big.add_(1.0)
        got = load_experts_fp8(w, H, I, DEV, stream)
        junk = [torch.full((H, I), float("nan"), device=DEV) for _ in range(8)]
        assert torch.equal(got, want)   # on the current stream, behind the load
        assert len(junk) == 8


def test_load_numpy_and_half():
    """Host arrays and other float types give the blobs of their fp32 values."""
    say("fp8 load types")
    H, I = 192, 128
    r = np.random.default_rng(5)
    w = [tuple(r.normal(0, 0.02, s).astype(np.float16) for s in ((I, H), (I, H), (H, I)))
         for _ in range(3)]
    want = load_experts_fp8([tuple(m.astype(np.float32) for m in e) for e in w], H, I, DEV)
    assert torch.equal(load_experts_fp8(w, H, I, DEV), want)
    views = [tuple(torch.from_numpy(m).to(DEV).t().contiguous().t() for m in e) for e in w]
    assert torch.equal(load_experts_fp8(views, H, I, DEV), want)
