"""What the layers with score routing and FP8 experts refuse before any call
into the library; no GPU is touched."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
from int4_weight_only_router_amd.layer import MoELayer, ScoreRouting, load_experts_fp8

H, I = 128, 64


def _expert(*shapes):
    return tuple(np.zeros(s, np.float32) for s in shapes)


@pytest.mark.parametrize("bad", [
    _expert((H, I), (I, H), (H, I)),            # as many elements, transposed
    _expert((I, H), (I, H), (I, H)),
    _expert((I // 2, H), (I, H), (H, I)),       # a shard: fewer elements than the kernel reads
    _expert((I, H), (I, H), (H, I - 1)),
    _expert((I * H,), (I, H), (H, I)),
    _expert((I, H), (I, H)),                    # a matrix short
    _expert((I, H), (I, H), (H, I), (H, I)),
    ()], ids=lambda w: "+".join("x".join(map(str, m.shape)) for m in w) or "none")
def test_load_refuses_other_shapes(bad):
    good = _expert((I, H), (I, H), (H, I))
    for weights in ([bad], [good, bad], iter([good, iter(bad)])):
        with pytest.raises(ValueError, match="expert [01]: matrices of shapes"):
            load_experts_fp8(weights, H, I, "cpu")


def _layer(fmt, routing):
    return MoELayer(256, 64, 4, 2, 64, torch.zeros((4, 256), dtype=torch.float16),
                    torch.zeros(4, dtype=torch.int64), device="cpu", fmt=fmt, routing=routing)


@pytest.mark.parametrize("fmt,routing", [(M.MOE_FMT_SYM, ScoreRouting()),
                                         (M.MOE_FMT_ZP, ScoreRouting()), (M.MOE_FMT_FP8, None),
                                         (M.MOE_FMT_FP8, ScoreRouting())])
def test_no_routing_from_logit_partials(fmt, routing):
    """The launch that routes from partials knows softmax top-k and INT4 blobs
    only: other layers are refused, not routed or read as what they are not."""
    lay, plain = _layer(fmt, routing), _layer(M.MOE_FMT_SYM, None)
    b, x, parts = lay.buffers(1), torch.zeros((1, 256), dtype=torch.float16), torch.zeros(1)
    with pytest.raises(ValueError):
        lay.experts_routed(x, b, parts)
    with pytest.raises(ValueError):
        lay.logit_partials(x, parts)
    with pytest.raises(ValueError):
        plain.combine_partials_next(plain.buffers(1), lay, parts)
