"""What the layers with score routing and FP8 experts refuse before any call
into the library; no GPU is touched."""
import numpy as np
import pytest

from int4_weight_only_router_amd.layer import load_experts_fp8

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
