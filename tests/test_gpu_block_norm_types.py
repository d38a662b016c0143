"""Ends and starts of blocks of which one has no weights, next to fp32 and fp16 ones."""
import pytest
import torch

import int4_weight_only_router_amd as M
from int4_weight_only_router_amd.layer import BlockNorms, block_norm
from tests import block_util as B
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
STEPS = 64   # as in test_gpu_block_norm


@pytest.mark.parametrize("t", [torch.float16, torch.float32])
@pytest.mark.parametrize("ends,starts", [(True, False), (False, True), (False, False), (True, True)])
@pytest.mark.parametrize("T,H", [(1, 256), (5, 1000)])
def test_weights_on_one_side(T, H, ends, starts, t):
    g = torch.Generator().manual_seed(T + H)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    w = lambda: (1.0 + 0.1 * r(H)).to(DEV, t)  # noqa: E731
    y, h = r(T, H).half().to(DEV), r(T, H).half().to(DEV)
    end = BlockNorms(post=True, post_w=w() if ends else None, post_b=w() if ends else None, scale=0.5)
    start = BlockNorms(w() if starts else None, w() if starts else None)
    out, n = torch.empty_like(h), torch.empty_like(h)
    block_norm(y, h, end, start, out, n)
    v = lambda x: None if x is None else x.cpu().double()  # noqa: E731
    c = dict(kind="rms", post=True, scale=0.5, eps=1e-5, offset=False)
    a = dict(y=v(y), residual=v(h), gate=None, post_w=v(end.post_w), post_b=v(end.post_b),
             pre_w=v(start.pre_w), pre_b=v(start.pre_b))
    for got, want, size in zip((out, n), B.block_norm_ref(c, a), B.block_norm_sizes(c, a)):
        assert ((v(got) - want).abs() <= 2.0 ** -11 * want.abs() + STEPS * B.U * size + 1e-7).all()
    assert end.w_dtype == (M.MOE_DTYPE_F32 if ends and t == torch.float32 else M.MOE_DTYPE_F16)
