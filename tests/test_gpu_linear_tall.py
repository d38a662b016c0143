"""A narrow product so tall that only wide tiles fit a launch, with rows beyond 2^31
elements and 2^32 bytes."""
import pytest
import torch

import int4_weight_only_router_amd as M
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [8, 3])
def test_tall(n):
    m, k = (1 << 28) + 5, 8
    say("linear %dx%dx%d" % (m, n, k))
    x = torch.empty((m, k), dtype=torch.float16, device=DEV)
    step = 1 << 24
    for r in range(0, m, step):   # whole numbers: every sum below is exact
        x[r:r + step] = torch.randint(-8, 9, x[r:r + step].shape, device=DEV, dtype=torch.int8)
    w = torch.randint(-8, 9, (n, k), device=DEV).half()
    out = torch.full((m, n), -3.0, dtype=torch.float16, device=DEV)
    nb = M.moe_linear_f16_workspace_bytes(m, n, k)
    assert nb == 0
    M.moe_linear_f16(x, k, w, k, None, M.MOE_ACT_NONE, None, 0, m, n, k, out, M.MOE_DTYPE_F16, n)
    for r in range(0, m, step):
        want = sum(x[r:r + step, j:j + 1].float() * w[:, j].float() for j in range(k))
        assert torch.equal(out[r:r + step].float(), want)
