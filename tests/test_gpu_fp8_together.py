"""FP8 layers and score routing in company: on two streams at once, with one
set of buffers for a whole stack, and without tokens."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
from int4_weight_only_router_amd.layer import ScoreRouting, stack_forward
from tests import test_gpu_fp8_layer as L
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
H, I, E, k = 512, 128, 24, 3


def _stack():
    r = np.random.default_rng(2)
    sig = ScoreRouting(M.MOE_SCORE_SIGMOID, None, 4, 2, True, 1.5)
    odd = ScoreRouting(M.MOE_SCORE_SOFTMAX, None, 8, 5, False, 2.0)
    return [L._layer(r, H, I, E, k, how) for how in (sig, None, odd, None, None, sig)], r


@pytest.mark.parametrize("fuse", [False, True])
@pytest.mark.parametrize("T", [1, 3, 5, 40, 200])
def test_shared_buffers(T, fuse):
    """Every layer of a stack on the same buffers (routing arrays, workspaces,
    y), softmax and score layers in turn, twice: the bits of separate ones."""
    say("fp8 stack on shared buffers T=%d fuse=%d" % (T, fuse))
    layers, r = _stack()
    acts = lambda x: [x] + [torch.full((T, H), -7.0, dtype=torch.float16, device=DEV)   # noqa: E731
                            for _ in layers]
    one = layers[0].buffers(T)
    for _ in range(2):
        x = torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV)
        want, got = acts(x), acts(x)
        stack_forward(layers, [lay.buffers(T) for lay in layers], want, fuse=fuse)
        stack_forward(layers, [one] * len(layers), got, fuse=fuse)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 7, 90])
def test_two_streams_at_once(T):
    """Two batches through the same layers on two streams, each with buffers of
    its own, many passes in flight: the bits of one after the other."""
    say("fp8 layers on two streams T=%d" % T)
    layers, r = _stack()
    layers = [lay for lay in layers if lay.routing is not None]
    xs = [torch.from_numpy(r.normal(0, 1, (T, H)).astype(np.float16)).to(DEV) for _ in range(2)]

    def passes(x, bufs, out, stream, n):
        for _ in range(n):
            for lay, b, o in zip(layers, bufs, out):
                lay.forward(x, b, residual=x, out=o, stream=stream)
    make = lambda: ([lay.buffers(T) for lay in layers],   # noqa: E731
                    [torch.empty((T, H), dtype=torch.float16, device=DEV) for _ in layers])
    want = [make() for _ in xs]
    for x, (b, o) in zip(xs, want):
        passes(x, b, o, None, 1)
    got, streams = [make() for _ in xs], [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, (b, o), s in zip(xs, got, streams):
            passes(x, b, o, s, 5)
    torch.cuda.synchronize()
    for (_, a), (_, b) in zip(want, got):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_no_tokens():
    say("fp8 layer T=0")
    layers, _ = _stack()
    for lay in layers[:3]:
        b = lay.buffers(0)
        b.y.fill_(-7.0)
        out = lay.forward(torch.empty((0, H), dtype=torch.float16, device=DEV), b)
        torch.cuda.synchronize()
        assert out.shape == (0, H) and not bool(b.counts.any()) and not bool(b.offsets.any())
        assert bool((b.y == -7.0).all())
