"""One workspace, made for the largest batch, for every smaller one."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _w4
from tests._gpu import announce
from tests.test_gpu_moe import weights_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_workspace(dtype):
    g = np.random.default_rng(11)
    hidden, inner, experts, top_k, most = 512, 512, 48, 4, 200
    up, down = (w.device()[:2] for w in weights_of(_w4.MX, experts, hidden, inner, g))
    router = torch.from_numpy(g.standard_normal((experts, hidden))).float().cuda()
    xs = torch.from_numpy(g.standard_normal((most, hidden))).to(dtype).cuda()
    lib = fp4.lib()
    code = fp4.BF16 if dtype == torch.bfloat16 else fp4.F32
    space = torch.empty(max(
        lib.fp4_moe_route_workspace_bytes(most, hidden, experts),
        lib.fp4_moe_experts_workspace_bytes(fp4._moe_weights(fp4.MXFP4, up, down, 0), fp4.MXFP4,
                                            most, top_k, code)), dtype=torch.uint8, device="cuda")
    for tokens in (200, 1, 16, 33, 48, 64, 65, 100, 112, 113, 128, 199):
        announce(f"one workspace, {tokens} tokens, {dtype}")
        x = xs[:tokens]
        space.fill_(255)
        ids, w = fp4.moe_route(x, router, top_k, workspace=space)
        fresh = fp4.moe_route(x, router, top_k)
        assert torch.equal(ids, fresh[0]) and torch.equal(w, fresh[1])
        space.fill_(255)
        y = fp4.moe_experts(fp4.MXFP4, x, ids, w, up, down, workspace=space)
        assert torch.equal(y, fp4.moe_experts(fp4.MXFP4, x, ids, w, up, down))
