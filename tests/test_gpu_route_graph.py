"""Captured selections whose groups do not fall on whole power-of-two runs of
lanes (their keys go through dynamic LDS), captured as the first call of their
kernel and over several replays with eager calls between."""
import numpy as np
import pytest
import torch

import int4_weight_only_router_amd as M
from tests import fp8_util as R
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,G,keep", [
    (1, 60, 4, 6, 3), (5, 60, 4, 6, 3), (16, 500, 10, 10, 4), (777, 60, 4, 6, 3),
    (40, 768, 9, 3, 2), (300, 130, 5, 2, 1), (9, 1000, 3, 8, 2)])
def test_captured_odd_groups(T, E, k, G, keep, dtype):
    say("select graph T=%d E=%d groups=%d/%d %s" % (T, E, keep, G, dtype))
    dt = {torch.float32: M.MOE_DTYPE_F32, torch.float16: M.MOE_DTYPE_F16,
          torch.bfloat16: M.MOE_DTYPE_BF16}[dtype]
    r = np.random.default_rng(T + E)
    buf = torch.zeros((T, E), dtype=dtype, device=DEV)
    nws = M.moe_route_select_workspace_bytes(T, k, E)

    def outputs():
        i32 = lambda m: torch.zeros(m, dtype=torch.int32, device=DEV)   # noqa: E731
        return (i32(T * k), torch.zeros(T * k, device=DEV), i32(E), i32(E + 1), i32(T * k),
                i32(T * k), torch.zeros(max(nws, 1), dtype=torch.uint8, device=DEV))

    def call(o):
        M.moe_route_select_permute(buf, dt, E, None, T, E, k, M.MOE_SCORE_SIGMOID, G, keep,
                                   M.MOE_GROUP_TOP2 | M.MOE_RENORM, 1.5, *o, nws)
    held, eager = outputs(), outputs()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(held)
    for _ in range(3):
        buf.copy_(torch.from_numpy(r.normal(0, 1, (T, E)).astype(np.float32)))
        g.replay()
        call(eager)
        torch.cuda.synchronize()
        ri, rw = R.select(buf.float().cpu().numpy(), None, k, "sigmoid", G, keep, True, True, 1.5)
        want = (ri.reshape(-1),) + tuple(R.grouping(ri, E))
        for o in (held, eager):
            w = o[1].cpu().numpy().reshape(T, k)
            assert np.all(np.abs(w - rw) <= 2 * R.U32 * np.abs(rw) + 2.0 ** -149)
            for a, b in zip((o[0],) + o[2:6], want):
                assert np.array_equal(a.cpu().numpy(), b)
