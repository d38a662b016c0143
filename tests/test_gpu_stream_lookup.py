"""The stream that a call without one takes is torch's current stream, by the
raw lookup and by the public one."""
import pytest
import torch

from int4_weight_only_router_amd import _abi as A
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [True, False])
def test_current_stream(raw, monkeypatch):
    say("stream lookup raw=%d" % raw)
    monkeypatch.setattr(A, "_raw_stream", None)
    if not raw:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    side, other = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    assert A._s(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert A._s(None) == side.cuda_stream
        with torch.cuda.stream(other):
            assert A._s(None) == other.cuda_stream
        assert A._s(None) == side.cuda_stream
    assert A._s(None) == torch.cuda.current_stream().cuda_stream
    assert A._s(side) == side.cuda_stream and A._s(5) == 5
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):   # captures on a stream of its own
        held = A._s(None)
        assert held == torch.cuda.current_stream().cuda_stream
        torch.zeros(1, device=DEV).add_(1)
    assert held != torch.cuda.current_stream().cuda_stream
