"""The decoding layers in use: one after the other around the cache, each against
the definition in 64 bits on what it was given; in one graph; on streams side by side;
and at sizes past 32 bits."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _kv, _moe, _w4
from tests._gpu import announce
from tests.test_gpu_moe import check_experts, weights_of
from tests.test_gpu_norm_rotate import check as check_rotated, frequencies, reference

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, INNER, EXPERTS, TOP = 512, 8, 2, 128, 96, 12, 3


class Layer:
    """qkv -> norm and rotation -> cache -> attention -> output, then the experts."""

    def __init__(self, g):
        def plain(n, k):
            base = 126 + round(np.log2(0.6 * k ** -0.5))
            return _w4.Weight(_w4.MX, g.integers(0, 256, (n, k // 2)).astype(np.uint8),
                              g.integers(base, base + 3, (n, k // 32)).astype(np.uint8))
        self.qkv, self.out = plain((HEADS + 2 * KV) * DIM, HIDDEN), plain(HIDDEN, HEADS * DIM)
        self.qkv_packed = fp4.pack_mxfp4_operand(*self.qkv.device()[:2])
        self.out_rows = self.out.device()[:2]
        self.router = torch.from_numpy(g.standard_normal((EXPERTS, HIDDEN)) * HIDDEN ** -0.5).float()
        self.router_dev = self.router.cuda()
        self.up, self.down = weights_of(_w4.NV, EXPERTS, HIDDEN, INNER, g)
        self.up_dev, self.down_dev = self.up.device(), self.down.device()
        self.norms = torch.from_numpy(1 + 0.3 * g.standard_normal((2, DIM))).bfloat16()
        self.q_norm, self.k_norm = (w.contiguous().cuda() for w in self.norms)
        self.freq = frequencies(DIM)
        self.freq_dev = self.freq.cuda()
        self.cache = fp4.new_kv_cache(24, KV, 32, DIM, "cuda")

    def __call__(self, x, batch):
        """Every value on the way, by name."""
        n = (HEADS + 2 * KV) * DIM
        v = {"qkv": fp4.linear_w4_packed(fp4.MXFP4, x, self.qkv_packed, n)}
        heads = v["qkv"].view(x.shape[0], -1, DIM)
        v["q"], v["k"] = fp4.norm_rotate(heads[:, :HEADS], heads[:, HEADS:HEADS + KV], *batch[:2],
                                         self.freq_dev, self.q_norm, self.k_norm, check=False)
        fp4.kv_cache_write(self.cache, v["k"], heads[:, HEADS + KV:], *batch, check=False)
        v["o"] = fp4.kv_attention(v["q"], self.cache, *batch, check=False)
        v["h"] = x + fp4.linear_w4(fp4.MXFP4, v["o"].flatten(1), *self.out_rows)
        v["ids"], v["weights"] = fp4.moe_route(v["h"], self.router_dev, TOP)
        v["y"] = fp4.moe_experts(fp4.NVFP4, v["h"], v["ids"], v["weights"], self.up_dev,
                                 self.down_dev, check=False)
        return v


def product(x, w, roundings):
    """x times a weight, and the bound of its bf16 output's error."""
    x, values = x.double().cpu().numpy(), w.values()
    want = x @ values.T
    return want, (_w4.product_bound(roundings, np.abs(x) @ np.abs(values).T)
                  + 1.01 * 2.0 ** -8 * np.abs(want))


def batches(new, old, table):
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    lengths = [a + b for a, b in zip(new, old)]
    return cu, lengths, (i32(cu), i32(lengths), i32(table))


TABLE = [[5, 1, 9, 20], [2, 7, 0, 3], [11, 4, 6, 8]]


def test_one_after_the_other():
    g = np.random.default_rng(0)
    layer = Layer(g)
    old = [0, 0, 0]
    for new in ([70, 0, 33], [1, 5, 1], [1, 1, 1], [0, 30, 2]):
        announce(f"decoding layers, {new} new tokens after {old}")
        cu, lengths, batch = batches(new, old, TABLE)
        x = torch.from_numpy(g.standard_normal((cu[-1], HIDDEN))).bfloat16().cuda()
        v = {k: t.cpu() for k, t in layer(x, batch).items()}
        # at least four waves share K
        want, bound = product(x, layer.qkv, HIDDEN / 4 + 16)
        assert (np.abs(v["qkv"].double().numpy() - want) <= bound).all()
        pos = torch.cat([torch.arange(o, o + n) for n, o in zip(new, old)])
        heads = v["qkv"].view(cu[-1], -1, DIM)
        for got, rows, norm in ((v["q"], heads[:, :HEADS], layer.norms[0]),
                                (v["k"], heads[:, HEADS:HEADS + KV], layer.norms[1])):
            check_rotated(got, *reference(rows, norm, pos, layer.freq, 1e-6, False), torch.bfloat16)

        starts = np.concatenate([[0], np.cumsum(lengths)]).tolist()
        whole = (torch.tensor(starts, dtype=torch.int32, device="cuda"), *batch[1:])
        k, values = fp4.kv_cache_read(layer.cache, *whole, starts[-1], out_dtype=torch.float32)
        seen = Values(k.double().cpu().numpy(), values.double().cpu().numpy())
        q = v["q"].double().numpy()
        want, _, weight, reach = _kv.attention(seen, q, cu, lengths, [[s] for s in starts], DIM ** -0.5)
        bound, _ = _kv.tolerance(weight, reach, want, max(lengths), DIM, True)
        assert (np.abs(v["o"].double().numpy() - want) <= bound).all()

        want, bound = product(v["o"].flatten(1), layer.out, HEADS * DIM / 4 + 16)
        # bf16 once after the product, again after x is added
        want = want + x.double().cpu().numpy()
        bound = bound + 1.01 * 2.0 ** -8 * (np.abs(want) + bound)
        assert (np.abs(v["h"].double().numpy() - want) <= bound).all()
        ids, weights = _moe.choose(v["h"].double().numpy() @ layer.router.double().numpy().T, TOP, True)
        assert np.array_equal(v["ids"].numpy(), ids)
        assert np.allclose(v["weights"].double().numpy(), weights, rtol=2.0 ** -24 + 1e-9, atol=0)
        check_experts(fp4.NVFP4, v["h"], ids, v["weights"].numpy(), layer.up, layer.down)
        old = lengths


class Values:
    """What the reference needs of a cache: one sequence's values."""

    def __init__(self, k, v):
        self.kv = k, v

    def sequence(self, half, table, length):
        return self.kv[half][table[0]:table[0] + length]


def test_one_graph():
    """A step captured once serves every following token: lengths and rows are data."""
    g = np.random.default_rng(1)
    eager, layer = Layer(g), Layer(np.random.default_rng(1))
    x = torch.zeros(3, HIDDEN, dtype=torch.bfloat16, device="cuda")
    _, _, batch = batches([1, 1, 1], [0, 0, 0], TABLE)
    layer(x, batch)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v = layer(x, batch)
    for step in range(5):
        _, _, fresh = batches([1, 1, 1], [step, step, step], TABLE)
        x.copy_(torch.from_numpy(g.standard_normal((3, HIDDEN))))
        batch[1].copy_(fresh[1])
        graph.replay()
        torch.cuda.synchronize()
        want = eager(x, fresh)
        for name in want:
            assert torch.equal(v[name], want[name]), (step, name)


@pytest.mark.parametrize("tokens", [1, 40])
def test_side_by_side(tokens):
    """Calls on two streams at once, each with its own scratch; then two graphs on one
    stream that share it."""
    g = np.random.default_rng(tokens)
    up, down = weights_of(_w4.MX, 16, 256, 512, g)
    u, d = up.device()[:2], down.device()[:2]
    dev = lambda a, dtype: torch.from_numpy(a).to(dtype).cuda()
    xs = [dev(g.standard_normal((tokens, 256)), torch.bfloat16) for _ in range(2)]
    router = dev(g.standard_normal((16, 256)) / 16, torch.float32)

    def step(x, space=None, route_space=None):
        ids, w = fp4.moe_route(x, router, 4, workspace=route_space)
        return fp4.moe_experts(fp4.MXFP4, x, ids, w, u, d, workspace=space, check=False)

    want = [step(x).clone() for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for s, x, outs in zip(streams, xs, got):
            with torch.cuda.stream(s):
                outs.append(step(x))
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)
    need = fp4.lib().fp4_moe_experts_workspace_bytes(
        fp4._moe_weights(fp4.MXFP4, u, d, 0), fp4.MXFP4, tokens, 4, fp4.BF16)
    spaces = (torch.empty(need, dtype=torch.uint8, device="cuda"),
              torch.empty(fp4.lib().fp4_moe_route_workspace_bytes(tokens, 256, 16),
                          dtype=torch.uint8, device="cuda"))
    graphs, outs = [], []
    for x in xs:
        step(x, *spaces)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(x, *spaces))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for x, o in zip(xs, outs):
            assert torch.equal(o, step(x))
            x.normal_()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,experts,top_k", [(130, 64, 32), (64, 1024, 32), (70, 33, 32)])
def test_many_experts_a_token(tokens, experts, top_k, dtype):
    """Plans of thousands of pairs."""
    announce(f"moe_experts {tokens} of {experts}, {top_k} a token, {dtype}")
    g = np.random.default_rng(experts)
    up, down = weights_of(_w4.MX, experts, 32, 32, g)
    ids = np.argsort(g.random((tokens, experts)), axis=1)[:, :top_k]
    ids[g.random(ids.shape) < 0.1] = -1
    weights = g.random((tokens, top_k)).astype(np.float32)
    x = torch.from_numpy(g.standard_normal((tokens, 32))).to(dtype)
    check_experts(_w4.MX, x, ids, weights, up, down)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,tokens,hidden,inner,experts,top_k", [
    (_w4.MX, 8, 64, 96, 2, 2), (_w4.NV, 30, 96, 544, 2, 2), (_w4.MX, 64, 32, 2048, 16, 2),
    (_w4.NV, 21, 48, 1040, 4, 3), (_w4.MX, 64, 4096, 512, 3, 1), (_w4.NV, 100, 256, 512, 32, 4),
    (_w4.MX, 4, 64, 8192, 2, 1)])
def test_shared_passes(fmt, tokens, hidden, inner, experts, top_k, dtype):
    """Experts with many tokens each, and rows so few that workgroups share them."""
    announce(f"moe_experts {fmt} {tokens} {hidden} {inner} {experts} {top_k} {dtype}")
    g = np.random.default_rng(inner + tokens)
    up, down = weights_of(fmt, experts, hidden, inner, g)
    ids = np.argsort(g.random((tokens, experts)), axis=1)[:, :top_k]
    ids[0] = -1
    weights = g.random((tokens, top_k)).astype(np.float32)
    x = torch.from_numpy(g.standard_normal((tokens, hidden))).to(dtype)
    check_experts(fmt, x, ids, weights, up, down)


def test_shared_passes_captured():
    g = np.random.default_rng(9)
    up, down = weights_of(_w4.MX, 4, 128, 1024, g)
    u, d = up.device()[:2], down.device()[:2]
    x = torch.randn(40, 128, device="cuda").bfloat16()
    ids = torch.randint(-1, 4, (40, 2), dtype=torch.int32, device="cuda")
    weights = torch.rand(40, 2, device="cuda")
    out = torch.empty(40, 128, device="cuda")

    def step():
        return fp4.moe_experts(fp4.MXFP4, x, ids, weights, u, d, out=out, check=False)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        x.normal_()
        ids.random_(-1, 4)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, fp4.moe_experts(fp4.MXFP4, x, ids, weights, u, d,
                                                out_dtype=torch.float32))


@pytest.mark.parametrize("fmt,m,n,k", [
    (_w4.MX, 17, 31, 96), (_w4.NV, 64, 8192, 80), (_w4.MX, 33, 28700, 544), (_w4.NV, 130, 4097, 528),
    (_w4.MX, 64, 28672, 1024), (_w4.MX, 500, 1000, 224)])
def test_every_tile_of_many_tokens(fmt, m, n, k):
    """Whole-number activations: sums are exact, so every tile's is the same."""
    announce(f"linear_w4 {fmt} {m} x {n} x {k}")
    g = np.random.default_rng(n)
    w = _w4.exact_weight(fmt, (n, k), g)
    x = g.integers(-8, 9, (m, k)).astype(np.float32)
    want = torch.from_numpy(x.astype(np.float64) @ w.values().T * w.factor()).float()
    codes, scales, s_g = w.device()
    for dtype in (torch.bfloat16, torch.float32):
        xd = torch.from_numpy(x).to(dtype).cuda()
        got = fp4.linear_w4(fmt, xd, codes, scales, s_g, out_dtype=torch.float32)
        assert torch.equal(got.cpu(), want)


# ---- past 32 bits ---------------------------------------------------------------
def random_bytes(*shape):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("m", [1, 20])
def test_weights_of_more_than_2_31_bytes(m):
    announce(f"linear_w4 {m} x 150016 x 32768")
    n, k = 150016, 32768
    codes = random_bytes(n, k // 2)
    scales = torch.randint(110, 124, (n, k // 32), dtype=torch.uint8, device="cuda")
    x = torch.randn(m, k, device="cuda").bfloat16()
    got = fp4.linear_w4(fp4.MXFP4, x, codes, scales)
    # four waves or more share K; another N may have another order of sums
    x = x.double().cpu().numpy()
    for at in (0, 131072 - 256, n - 256):
        part = slice(at, at + 256)
        values = _w4.Weight(_w4.MX, codes[part].cpu().numpy(), scales[part].cpu().numpy()).values()
        want = x @ values.T
        bound = (_w4.product_bound(k / 4 + 16, np.abs(x) @ np.abs(values).T)
                 + 1.01 * 2.0 ** -8 * np.abs(want))
        err = np.abs(got[:, part].double().cpu().numpy() - want)
        assert (err <= bound).all()
        # the sums' errors as a whole are far below that: the output's rounding
        assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(want)


def test_outputs_of_more_than_2_31_elements():
    announce("linear_w4 70000 x 32800 x 32")
    m, n = 70000, 32800
    codes = random_bytes(n, 16)
    scales = torch.randint(120, 130, (n, 1), dtype=torch.uint8, device="cuda")
    x = torch.randn(m, 32, device="cuda").bfloat16()
    got = fp4.linear_w4(fp4.MXFP4, x, codes, scales)
    for at in (0, 65536, m - 64):
        part = slice(at, at + 64)
        assert torch.equal(got[part], fp4.linear_w4(fp4.MXFP4, x[part], codes, scales))


def test_experts_of_more_than_2_31_bytes():
    announce("moe_experts of 20 x 8192 x 14336")
    experts, hidden, inner = 20, 8192, 14336

    def make(rows, k):
        return (random_bytes(experts, rows, k // 2),
                torch.randint(117, 121, (experts, rows, k // 32), dtype=torch.uint8, device="cuda"))
    up, down = make(2 * inner, hidden), make(hidden, inner)
    x = torch.randn(3, hidden, device="cuda").bfloat16()
    w = torch.ones(3, 1, device="cuda")
    for e in (0, 18, 19):
        ids = torch.full((3, 1), e, dtype=torch.int32, device="cuda")
        got = fp4.moe_experts(fp4.MXFP4, x, ids, w, up, down)
        alone = [tuple(t[e:e + 1].contiguous() for t in part) for part in (up, down)]
        assert torch.equal(got, fp4.moe_experts(fp4.MXFP4, x, 0 * ids, w, *alone))
        assert got.isfinite().all() and (got != 0).any()


def test_many_tokens_of_a_router():
    announce("moe_route 300000 x 8 of 1024")
    tokens = 300000
    x = torch.randn(tokens, 8, device="cuda")
    router = torch.randn(1024, 8, device="cuda")
    ids, w = fp4.moe_route(x, router, 4)
    for at in (0, 262144, tokens - 64):
        part = slice(at, at + 64)
        some, share = fp4.moe_route(x[part], router, 4)
        assert torch.equal(ids[part], some) and torch.equal(w[part], share)
