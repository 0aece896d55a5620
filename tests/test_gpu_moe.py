"""The router's choice and the experts' products, against 64 bits."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _moe, _w4
from tests._gpu import announce

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- router -------------------------------------------------------------------
def check_route(x, router, top_k, renormalize):
    logits = x.double().numpy() @ router.double().numpy().T
    ids, p = _moe.choose(logits, top_k, renormalize)
    got, w = fp4.moe_route(x.cuda(), router.cuda(), top_k, renormalize)
    assert got.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(got.cpu().numpy(), ids)
    w = w.cpu().double().numpy()
    # 64-bit sums and exponentials, rounded once
    assert np.allclose(w, p, rtol=2.0 ** -24 + 1e-9, atol=1e-45, equal_nan=True)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("router", list(DTYPES))
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,hidden,experts,top_k", [
    (1, 8, 1, 1), (1, 2048, 64, 4), (3, 40, 5, 5), (15, 104, 17, 2), (16, 128, 16, 1),
    (17, 136, 65, 8), (33, 1000, 100, 6), (64, 512, 256, 8), (70, 264, 257, 32), (5, 96, 1024, 32),
    (2, 8192, 33, 3), (300, 64, 20, 2)])
def test_route(tokens, hidden, experts, top_k, dtype, router, renormalize):
    announce(f"moe_route {tokens} {hidden} {experts} {top_k} {dtype} {router} {renormalize}")
    g = torch.Generator().manual_seed(tokens * 31 + experts)
    x = torch.randn(tokens, hidden, generator=g).to(DTYPES[dtype])
    r = (torch.randn(experts, hidden, generator=g) * hidden ** -0.5).to(DTYPES[router])
    check_route(x, r, top_k, renormalize)


def test_equal_logits():
    """Of equal ones the lower id; also where a token has nothing but equal ones."""
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-3, 4, (20, 64), generator=g).float()
    x[7] = 0
    rows = torch.randint(-2, 3, (9, 64), generator=g).float()
    r = rows[torch.randint(0, 9, (200,), generator=g)]  # many rows alike
    check_route(x, r, 12, True)
    check_route(x, r, 12, False)


def test_logits_next_to_each_other():
    """A difference that fp32 sums would lose decides."""
    x = torch.ones(1, 4096)
    r = torch.ones(3, 4096)
    r[1, 4095] += 2.0 ** -20
    r[2, 0] += 2.0 ** -19
    got, _ = fp4.moe_route(x.cuda(), r.cuda(), 3)
    assert got.cpu().tolist() == [[2, 1, 0]]


def test_logits_that_are_not_finite():
    x = torch.zeros(4, 64)
    x[0, 0], x[1, 1], x[2] = 1, 1, float("nan")
    r = torch.zeros(6, 64)
    r[0, 0], r[1, 0], r[3, 0] = float("nan"), float("-inf"), 2.0
    r[2, 1] = float("inf")
    # 0 * inf and 0 * NaN are NaN: rows 0, 1 of every token but 0, row 2 of every one but 1
    check_route(x, r, 6, True)
    check_route(x[:1].contiguous(), r[3:].contiguous(), 2, False)


def test_route_captured_and_given_outputs():
    g = torch.Generator().manual_seed(9)
    xs = [torch.randn(6, 256, generator=g).cuda() for _ in range(3)]
    r = torch.randn(40, 256, generator=g).cuda()
    x = xs[0].clone()
    out = (torch.empty(6, 4, dtype=torch.int32, device="cuda"), torch.empty(6, 4, device="cuda"))
    fp4.moe_route(x, r, 4, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4.moe_route(x, r, 4, out=out)
    for fresh in xs:
        x.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        ids, w = fp4.moe_route(fresh, r, 4)
        assert torch.equal(out[0], ids) and torch.equal(out[1], w)


# ---- experts ------------------------------------------------------------------
def weights_of(fmt, experts, hidden, inner, g, one_scale=False):
    def make(rows, k):
        codes = g.integers(0, 256, (experts, rows, k // 2)).astype(np.uint8)
        at = (experts, rows, k // _w4.BLOCK[fmt])
        if fmt == _w4.MX:
            base = 126 + round(np.log2(0.6 * k ** -0.5))
            return _w4.Weight(fmt, codes, g.integers(base, base + 3, at).astype(np.uint8))
        scales = g.integers(0x50, 0x5F, at) + 128 * g.integers(0, 2, at)
        s_g = g.uniform(0.5, 2, experts) * 0.02 * k ** -0.5
        if one_scale:
            s_g[:] = s_g[0]
        return _w4.Weight(fmt, codes, scales.astype(np.uint8), s_g.astype(np.float32))
    return make(2 * inner, hidden), make(hidden, inner)


def run(fmt, x, ids, weights, up, down, one_scale=False, **how):
    dev = []
    for w in (up, down):
        codes, scales, s_g = w.device()
        dev.append((codes, scales) if s_g is None else (codes, scales,
                                                        s_g[:1] if one_scale else s_g))
    return fp4.moe_experts(fmt, x.cuda(), torch.from_numpy(ids).int().cuda(),
                           torch.from_numpy(weights).float().cuda(), *dev, **how)


def check_experts(fmt, x, ids, weights, up, down, one_scale=False):
    terms, act = (3, 2.0 ** -23) if x.dtype == torch.float32 else (1, 2.0 ** -17)
    want, bound = _moe.layer(x.double().numpy(), ids, weights, up, down, terms, act)
    got = run(fmt, x, ids, weights, up, down, one_scale).cpu()
    assert got.dtype == x.dtype
    bound = bound + 1.01 * _w4.output_eps(x.dtype) * np.abs(want) + 1e-37
    err = np.abs(got.double().numpy() - want)
    assert (err <= bound).all(), (err / bound).max()
    # a row's error as a whole is far below the worst case of each element
    eps = 2.0 ** -8 if x.dtype == torch.bfloat16 else 3e-6
    assert np.linalg.norm(err) <= eps * np.linalg.norm(want)


CASES = [  # tokens, hidden, inner, experts, top_k
    (1, 32, 32, 1, 1), (1, 2048, 768, 64, 4), (2, 288, 160, 3, 2), (7, 1056, 480, 20, 3),
    (15, 256, 512, 8, 2), (16, 512, 256, 128, 8), (17, 160, 96, 4, 4), (33, 544, 288, 40, 6),
    (64, 256, 128, 16, 4), (65, 96, 64, 5, 2), (150, 64, 96, 200, 8), (3, 4096, 64, 6, 2),
    (5, 64, 4128, 6, 2)]
NV_CASES = [(3, 48, 16, 4, 2), (7, 1040, 496, 20, 3), (40, 80, 112, 12, 3), (1, 16, 272, 2, 1)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("fmt,tokens,hidden,inner,experts,top_k",
                         [(f, *c) for f in (_w4.MX, _w4.NV) for c in CASES]
                         + [(_w4.NV, *c) for c in NV_CASES])
def test_experts(fmt, tokens, hidden, inner, experts, top_k, dtype):
    announce(f"moe_experts {fmt} {tokens} {hidden} {inner} {experts} {top_k} {dtype}")
    g = np.random.default_rng(tokens * 131 + hidden + inner)
    up, down = weights_of(fmt, experts, hidden, inner, g)
    ids = np.argsort(g.random((tokens, experts)), axis=1)[:, :top_k]
    weights = g.random((tokens, top_k)).astype(np.float32)
    x = torch.from_numpy(g.standard_normal((tokens, hidden))).to(DTYPES[dtype])
    check_experts(fmt, x, ids, weights, up, down)


@pytest.mark.parametrize("tokens", [5, 20, 70])
@pytest.mark.parametrize("fmt", [_w4.MX, _w4.NV])
def test_ids_of_all_kinds(fmt, tokens):
    """None, the same one twice or in every slot, all tokens to one expert, rows
    without any, weights of zero and below."""
    g = np.random.default_rng(tokens)
    hidden, inner, experts, top_k = 96, 64, 9, 4
    up, down = weights_of(fmt, experts, hidden, inner, g, one_scale=True)
    ids = g.integers(-1, experts, (tokens, top_k))
    ids[0] = -1
    ids[1] = 5
    ids[2] = [7, -1, 7, 3]
    ids[-1] = -1
    weights = g.standard_normal((tokens, top_k)).astype(np.float32)
    weights[3] = 0
    x = torch.from_numpy(g.standard_normal((tokens, hidden))).float()
    check_experts(fmt, x, ids, weights, up, down, one_scale=True)
    ids[:] = 4
    check_experts(fmt, x, ids, weights, up, down, one_scale=True)
    ids[:] = -1
    assert (run(fmt, x, ids, weights, up, down) == 0).all()


@pytest.mark.parametrize("tokens", [3, 40])
@pytest.mark.parametrize("experts", [4, 300])  # a workgroup for each expert, for each slot
def test_ids_out_of_range(tokens, experts):
    g = np.random.default_rng(1)
    up, down = weights_of(_w4.MX, experts, 64, 32, g)
    ids = g.integers(0, experts, (tokens, 2))
    bad = ids.copy()
    ids[1, 1], bad[1, 1] = -1, experts
    ids[2, 0], bad[2, 0] = -1, -2 ** 31
    weights = g.random((tokens, 2)).astype(np.float32)
    x = torch.from_numpy(g.standard_normal((tokens, 64))).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = run(_w4.MX, x, ids, weights, up, down, check=False, status=status)
    assert status.item() == 0
    got = run(_w4.MX, x, bad, weights, up, down, check=False, status=status)
    assert status.item() == fp4.FLAG_EXPERT_INDEX
    assert torch.equal(got, want)
    with pytest.raises(ValueError):
        run(_w4.MX, x, bad, weights, up, down)
    run(_w4.MX, x, ids, weights, up, down)


@pytest.mark.parametrize("tokens", [4, 33])
@pytest.mark.parametrize("fmt", [_w4.MX, _w4.NV])
def test_what_is_not_finite_stays_with_its_tokens(fmt, tokens):
    g = np.random.default_rng(2)
    hidden, inner, experts = 128, 96, 6
    up, down = weights_of(fmt, experts, hidden, inner, g)
    ids = np.stack([np.arange(tokens) % 2, 2 + np.arange(tokens) % 2], 1)
    weights = g.random((tokens, 2)).astype(np.float32)
    x = torch.from_numpy(g.standard_normal((tokens, hidden))).bfloat16()
    want = run(fmt, x, ids, weights, up, down)
    # experts that nobody names
    nan = 255 if fmt == _w4.MX else 127
    for w in (up, down):
        w.scales[4:] = nan
    assert torch.equal(run(fmt, x, ids, weights, up, down), want)
    # one that odd tokens name
    down.scales[1, 7] = nan
    got = run(fmt, x, ids, weights, up, down).cpu()
    assert torch.equal(got[0::2], want.cpu()[0::2])
    odd = got[1::2]
    assert odd[:, 7].isnan().all()
    odd[:, 7] = want.cpu()[1::2, 7]
    assert torch.equal(odd, want.cpu()[1::2])
    up.scales[1] = nan
    got = run(fmt, x, ids, weights, up, down).cpu()
    assert torch.equal(got[0::2], want.cpu()[0::2]) and got[1::2].isnan().all()
    # an activation reaches its own row
    up, down = weights_of(fmt, experts, hidden, inner, np.random.default_rng(2))
    x[2, 5] = float("nan")
    got = run(fmt, x, ids, weights, up, down).cpu()
    rest = [t for t in range(tokens) if t != 2]
    assert got[2].isnan().all() and torch.equal(got[rest], want.cpu()[rest])


def test_captured_with_given_buffers():
    """Other experts at every replay, and no tokens at all."""
    g = np.random.default_rng(3)
    hidden, inner, experts, tokens = 256, 128, 24, 10
    up, down = weights_of(_w4.MX, experts, hidden, inner, g)
    u, d = up.device()[:2], down.device()[:2]
    x = torch.randn(tokens, hidden, device="cuda")
    ids = torch.zeros(tokens, 3, dtype=torch.int32, device="cuda")
    weights = torch.rand(tokens, 3, device="cuda")
    need = fp4.lib().fp4_moe_experts_workspace_bytes(
        fp4._moe_weights(fp4.MXFP4, u, d, 0), fp4.MXFP4, tokens, 3, fp4.F32)
    space = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    how = dict(out=out, workspace=space, check=False)
    fp4.moe_experts(fp4.MXFP4, x, ids, weights, u, d, **how)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4.moe_experts(fp4.MXFP4, x, ids, weights, u, d, **how)
    for k in range(4):
        fresh = torch.randint(-1, experts, (tokens, 3), dtype=torch.int32, device="cuda")
        ids.copy_(fresh if k != 2 else torch.full_like(fresh, -1))
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, fp4.moe_experts(fp4.MXFP4, x, ids, weights, u, d))
    assert fp4.moe_experts(fp4.MXFP4, x[:0], ids[:0], weights[:0], u, d).shape == (0, hidden)
