"""A workspace for the largest batch of a mixture of experts serves every smaller one
(no GPU is needed, pointers are never dereferenced)."""
import os

import pytest

import mxfp4_block_amax_amd as fp4

pytestmark = pytest.mark.skipif(not os.path.exists(fp4.LIB_PATH), reason="libfp4.so not built")

COUNTS = [*range(1, 700), 1000, 1024, 1025, 4096, 4097, 5000, 100000, 2 ** 19]


def rising(sizes):
    return all(0 < a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("hidden,experts", [
    (8, 1), (64, 16), (2048, 64), (4096, 256), (4096, 17), (1000, 1024), (65536, 3), (65536, 130)])
def test_route(hidden, experts):
    sizes = [fp4.lib().fp4_moe_route_workspace_bytes(t, hidden, experts) for t in COUNTS]
    assert rising(sizes)
    assert all(s >= t * experts * 8 for t, s in zip(COUNTS, sizes))


@pytest.mark.parametrize("xt", [fp4.F32, fp4.BF16])
@pytest.mark.parametrize("fmt", [fp4.MXFP4, fp4.NVFP4])
@pytest.mark.parametrize("hidden,inner,experts,top_k", [
    (32, 32, 8, 1), (32, 4096, 8, 2), (64, 96, 8, 32), (512, 512, 16, 4), (2048, 768, 128, 8),
    (2048, 2816, 8, 2), (4096, 1536, 128, 8), (32, 65536, 4, 32)])
def test_experts(hidden, inner, experts, top_k, fmt, xt):
    w = fp4._pack_moe_weights(16, 16, 16, 16, 16, 16, hidden, inner, experts, 0)
    sizes = [fp4.lib().fp4_moe_experts_workspace_bytes(w, fmt, t, top_k, xt) for t in COUNTS]
    assert rising(sizes)
    assert all(s >= t * top_k * inner * 4 for t, s in zip(COUNTS, sizes))


def test_sizes_in_between():
    """The most that any smaller count needs, not more: a batch of its own takes no more
    than one token more would."""
    size = fp4.lib().fp4_moe_route_workspace_bytes
    assert size(112, 4096, 256) == size(113, 4096, 256) == 917504
    assert size(2 ** 19, 64, 1024) == 2 ** 19 * 1024 * 8
