"""Linear layers of few tokens with FP4 weights, against 64 bits."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _w4
from tests._gpu import announce

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def layer(layout, weight, x, **how):
    codes, scales, s_g = weight.device()
    if layout == "rows":
        return fp4.linear_w4(weight.fmt, x, codes, scales, s_g, **how)
    pack = fp4.pack_mxfp4_operand if weight.fmt == _w4.MX else fp4.pack_nvfp4_operand
    return fp4.linear_w4_packed(weight.fmt, x, pack(codes, scales), codes.shape[0], s_g, **how)


# every M that starts a tile of tokens or ends one, N off the tiles of rows, K that ends
# in each part of a unit of 256
ROWS = [(m, n, k) for m, n, k in
        [(1, 1, 32), (1, 31, 64), (2, 33, 96), (1, 512, 2048), (3, 100, 128), (15, 65, 160),
         (16, 32, 256), (17, 7, 288), (5, 129, 416), (31, 64, 480), (32, 50, 512), (33, 16, 544),
         (48, 40, 1184), (63, 35, 2016), (64, 34, 4096), (65, 33, 768), (130, 70, 1056),
         (1, 4100, 352), (4, 3, 16384)]]
ODD = [(1, 5, 16), (3, 40, 48), (16, 33, 112), (20, 17, 144), (1, 70, 272), (65, 35, 496),
       (2, 64, 4112)]  # NVFP4's blocks of 16
PACKED = [(1, 32, 512), (1, 1, 512), (7, 33, 1024), (16, 100, 1536), (17, 64, 512),
          (40, 31, 2560), (64, 70, 4096), (129, 65, 512), (1, 2000, 8192)]
CASES = ([(fmt, "rows", *s) for fmt in (_w4.MX, _w4.NV) for s in ROWS]
         + [(_w4.NV, "rows", *s) for s in ODD]
         + [(fmt, "packed", *s) for fmt in (_w4.MX, _w4.NV) for s in PACKED])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("fmt,layout,m,n,k", CASES)
def test_sums_that_fp32_holds(fmt, layout, m, n, k, dtype):
    """Whole-number activations: every partial sum is exact, so is the result."""
    announce(f"linear_w4 exact {fmt} {layout} {m}x{n}x{k} {dtype}")
    g = np.random.default_rng(m * 7919 + n * 31 + k)
    w = _w4.exact_weight(fmt, (n, k), g)
    x = g.integers(-8, 9, (m, k)).astype(np.float32)
    want = x.astype(np.float64) @ w.values().T * w.factor()
    xd = torch.from_numpy(x).to(DTYPES[dtype]).cuda()
    got = layer(layout, w, xd, out_dtype=torch.float32)
    assert got.dtype == torch.float32
    assert np.array_equal(got.cpu().numpy(), want)
    got = layer(layout, w, xd, out_dtype=torch.bfloat16)
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.float32).bfloat16())


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("fmt,layout,m,n,k", [
    (_w4.MX, "rows", 1, 100, 4096), (_w4.MX, "packed", 5, 100, 4096), (_w4.NV, "rows", 20, 50, 2064),
    (_w4.NV, "packed", 64, 33, 1024)])
def test_any_values(fmt, layout, m, n, k, dtype):
    announce(f"linear_w4 {fmt} {layout} {m}x{n}x{k} {dtype}")
    g = np.random.default_rng(k)
    w = _w4.wide_weight(fmt, (n, k), g)
    x = torch.from_numpy(g.standard_normal((m, k)) * 2.0 ** g.integers(-20, 20, (m, k)))
    x = x.to(DTYPES[dtype])
    values = w.values()
    want = x.double().numpy() @ values.T * w.factor()
    size = np.abs(x.double().numpy()) @ np.abs(values).T * w.factor()
    out = DTYPES[dtype]
    got = layer(layout, w, x.cuda()).cpu()
    assert got.dtype == out
    # at least four waves share K, and an activation has up to three terms; the
    # tensor scale and the output round once each
    terms = 3 if dtype == "fp32" else 1
    bound = (_w4.product_bound(terms * k / 4 + 16, size)
             + (2.0 ** -24 + 1.01 * _w4.output_eps(out)) * np.abs(want))
    err = np.abs(got.double().numpy() - want)
    assert (err <= bound).all(), (err / bound).max()


def test_all_bits_of_fp32():
    """One activation a row, all 24 bits of it: nothing of it is lost."""
    g = np.random.default_rng(3)
    k, n = 512, 64
    codes = g.integers(0, 8, (n, k // 2)) * 17  # both values of a byte alike
    w = _w4.Weight(_w4.MX, codes.astype(np.uint8), np.full((n, k // 32), 127, dtype=np.uint8))
    x = torch.zeros(16, k)
    at = torch.arange(16) * 31
    x[torch.arange(16), at] = torch.from_numpy(
        (g.integers(2 ** 23, 2 ** 24, 16) * 2.0 ** g.integers(-60, 60, 16)).astype(np.float32))
    want = x.double().numpy() @ w.values().T
    for layout in ("rows", "packed"):
        got = layer(layout, w, x.cuda()).cpu().double().numpy()
        # three products of at most 10 bits each at one place: two roundings
        assert (np.abs(got - want) <= 2 * 2.0 ** -23 * np.abs(want)).all()


@pytest.mark.parametrize("fmt", [_w4.MX, _w4.NV])
@pytest.mark.parametrize("layout", ["rows", "packed"])
def test_scale_bytes(fmt, layout):
    """Every scale byte: exact up to MXFP4's 252, NaN rows for NaN, and no others."""
    n, k = 256, 512
    codes = np.full((n, k // 2), 0x23, dtype=np.uint8)  # 1.5, 1, ..
    scales = np.full((n, k // _w4.BLOCK[fmt]), 0 if fmt == _w4.NV else 20, dtype=np.uint8)
    byte = np.arange(256)
    scales[:, 5] = byte
    w = _w4.Weight(fmt, codes, scales, None if fmt == _w4.MX else np.ones(1, dtype=np.float32))
    x = torch.zeros(3, k)
    first = 5 * _w4.BLOCK[fmt]
    x[1, first] = 1.0
    x[2, first + 1] = 2.0
    got = layer(layout, w, x.cuda(), out_dtype=torch.float32).cpu().numpy().T
    values = (_w4.E8M0 if fmt == _w4.MX else _w4.E4M3)[byte]
    nan = np.isnan(values)
    assert np.isnan(got[nan]).all() and not np.isnan(got[~nan]).any()
    fits = ~nan & ((byte <= 252) | (fmt == _w4.NV))
    assert (got[fits, 0] == 0).all()
    assert np.array_equal(got[fits, 1], values[fits] * 1.5)
    assert np.array_equal(got[fits, 2], values[fits] * 2)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_activations_that_are_not_finite(dtype):
    """They reach their own row, as the products say."""
    g = np.random.default_rng(1)
    n, k = 40, 640
    codes = g.integers(1, 8, (n, k // 2)) * 17  # no zeros, none negative
    w = _w4.Weight(_w4.MX, codes.astype(np.uint8), np.full((n, k // 32), 127, dtype=np.uint8))
    x = torch.ones(20, k)
    x[2, 100], x[3, 639], x[4, 0] = float("inf"), float("-inf"), float("nan")
    x[5, 7], x[5, 8] = float("inf"), float("-inf")
    x[17, 33] = torch.finfo(DTYPES[dtype]).max / 16
    got = layer("rows", w, x.to(DTYPES[dtype]).cuda(), out_dtype=torch.float32).cpu()
    assert (got[2] == float("inf")).all() and (got[3] == float("-inf")).all()
    assert got[4:6].isnan().all()
    rest = [i for i in range(20) if i not in (2, 3, 4, 5)]
    assert got[rest].isfinite().all()


def test_outputs_given_and_streams():
    g = np.random.default_rng(2)
    w = _w4.exact_weight(_w4.MX, (70, 256), g)
    x = torch.from_numpy(g.integers(-8, 9, (2, 3, 256)).astype(np.float32)).cuda()
    want = layer("rows", w, x)
    assert want.shape == (2, 3, 70)
    codes, scales, _ = w.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = torch.full((2, 3, 70), 7.0, device="cuda")
        assert fp4.linear_w4(fp4.MXFP4, x, codes, scales, out=out) is out
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    assert fp4.linear_w4(fp4.MXFP4, x[:0], codes, scales).shape == (0, 3, 70)


def test_captured():
    g = np.random.default_rng(4)
    w = _w4.exact_weight(_w4.NV, (200, 512), g)
    codes, scales, s_g = w.device()
    xs = [torch.from_numpy(g.integers(-8, 9, (4, 512)).astype(np.float32)).cuda() for _ in range(3)]
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    fp4.linear_w4(fp4.NVFP4, x, codes, scales, s_g)
    with torch.cuda.graph(graph):
        y = fp4.linear_w4(fp4.NVFP4, x, codes, scales, s_g)
    for fresh in xs:
        x.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, fp4.linear_w4(fp4.NVFP4, fresh, codes, scales, s_g))
