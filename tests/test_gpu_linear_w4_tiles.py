"""Linear layers of many tokens with FP4 weights: every tile, in both formats and both
layouts, through whole rounds of its main loop and what is left of K."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _w4, _w4_tiles
from tests._gpu import announce
from tests.test_gpu_linear_w4 import layer

pytestmark = pytest.mark.gpu

IDS = [f"{t}x{r}-{m}x{n}" for (t, r), m, n in _w4_tiles.CASES]


def k_of(fmt, layout):
    return _w4_tiles.PACKED_K if layout == "packed" else _w4_tiles.ROWS_K[_w4.BLOCK[fmt]]


@pytest.mark.parametrize("tile,m,n", _w4_tiles.CASES, ids=IDS)
@pytest.mark.parametrize("layout", ["rows", "packed"])
@pytest.mark.parametrize("fmt", [_w4.MX, _w4.NV])
def test_sums_that_fp32_holds(fmt, layout, tile, m, n):
    """Whole-number activations: every partial sum is exact (below 2^19, in steps of 2^-5
    at least), so is the result."""
    k = k_of(fmt, layout)
    announce(f"linear_w4 tile {tile} {fmt} {layout} {m}x{n}x{k}")
    g = np.random.default_rng(m * 7919 + n)
    w = _w4.exact_weight(fmt, (n, k), g)
    x = torch.from_numpy(g.integers(-8, 9, (m, k)).astype(np.float32))
    want = torch.from_numpy(x.double().numpy() @ w.values().T * w.factor()).float()
    xd = x.bfloat16().cuda()
    assert torch.equal(layer(layout, w, xd, out_dtype=torch.float32).cpu(), want)
    assert torch.equal(layer(layout, w, xd).cpu(), want.bfloat16())


@pytest.mark.parametrize("tile", list(_w4_tiles.TILES))
@pytest.mark.parametrize("layout", ["rows", "packed"])
@pytest.mark.parametrize("fmt", [_w4.MX, _w4.NV])
def test_what_is_not_finite(fmt, layout, tile):
    """NaN scale bytes reach their rows of the weight, whichever wave has them; infinite
    activations and NaN their own rows.  The rest is what it is without them."""
    m, n = _w4_tiles.TILES[tile][-1]
    k = k_of(fmt, layout)
    announce(f"linear_w4 tile {tile} {fmt} {layout} {m}x{n}x{k}, NaN and infinities")
    g = np.random.default_rng(n)
    w = _w4.exact_weight(fmt, (n, k), g)
    x = torch.from_numpy(g.integers(-8, 9, (m, k)).astype(np.float32)).bfloat16()
    want = layer(layout, w, x.cuda(), out_dtype=torch.float32).cpu()
    scales = w.scales.copy()
    block = _w4.BLOCK[fmt]
    bad_rows = [0, 17, 63, 64, 100, n - 33, n - 1]
    for i, row in enumerate(bad_rows):
        w.scales[row, [0, 40, k // block - 1, 16, k // block - 2, 100, 77][i]] = \
            255 if fmt == _w4.MX else (127 if i % 2 else 255)
    got = layer(layout, w, x.cuda(), out_dtype=torch.float32).cpu()
    rows = [i for i in range(n) if i not in bad_rows]
    assert got[:, bad_rows].isnan().all() and torch.equal(got[:, rows], want[:, rows])
    w.scales = scales
    for row, (at, value) in {0: (0, np.inf), 15: (k - 1, -np.inf), 16: (4100, np.nan),
                             m - 1: (2500, np.inf)}.items():
        x[row, at] = value
    got = layer(layout, w, x.cuda(), out_dtype=torch.float32).cpu()
    tokens = [i for i in range(m) if i not in (0, 15, 16, m - 1)]
    assert torch.equal(got[tokens], want[tokens]) and got[16].isnan().all()
    values = torch.from_numpy(w.values())
    for row, at, sign in ((0, 0, 1), (15, k - 1, -1), (m - 1, 2500, 1)):
        # infinity times the weight's value: its sign, NaN of zero
        assert torch.equal(got[row].nan_to_num(0, 1, -1), sign * values[:, at].sign().float())
        assert torch.equal(got[row].isnan(), values[:, at] == 0)


def test_captured():
    m, n = _w4_tiles.TILES[2, 2][1]
    g = np.random.default_rng(5)
    w = _w4.exact_weight(_w4.NV, (n, 1024), g)
    codes, scales, s_g = w.device()
    packed = fp4.pack_nvfp4_operand(codes, scales)
    x = torch.randn(m, 1024, device="cuda").bfloat16()

    def step():
        return (fp4.linear_w4(fp4.NVFP4, x, codes, scales, s_g),
                fp4.linear_w4_packed(fp4.NVFP4, x, packed, n, s_g))
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
