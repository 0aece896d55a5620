"""GPU tests of attention over the 8-bit key/value cache against its definition
in 64 bits, within bounds derived in tests/_kv.py (tolerance)."""
import math

import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _kv
from tests._gpu import announce

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def filled(new, before, heads, block, dim, seed=0, std=1.0):
    """A cache written with random sequences, the rest of it arbitrary bytes."""
    total = [n + b for n, b in zip(new, before)]
    cu, lengths, table, pages = _kv.layout(new, before, block, seed=seed)
    ref = _kv.Cache(pages, heads, block, dim, seed)
    g = np.random.default_rng(seed + 1)
    x = [g.standard_normal((sum(total), heads, dim)) * std for _ in range(2)]
    x[0][..., 3::32] *= 4
    ref.write(x, np.concatenate([[0], np.cumsum(total)]).tolist(), total, table)
    return ref, cu, lengths, table


def queries(tokens, heads, dim, dtype, seed):
    x = torch.randn(tokens, heads, dim, generator=torch.Generator().manual_seed(seed))
    return x.to(TYPES[dtype])


def check(ref, dev, q, cu, lengths, table, scale=None, **how):
    dim, bf16 = q.shape[2], q.dtype == torch.bfloat16
    scale = dim ** -0.5 if scale is None else scale
    want, lse, weight, reach = _kv.attention(ref, q.double().numpy(), cu, lengths, table, scale,
                                             **how)
    got, got_lse = fp4.kv_attention(q.cuda(), dev, *_kv.batch(fp4, cu, lengths, table),
                                    scale=scale, return_lse=True, **how)
    got, got_lse = got.double().cpu().numpy(), got_lse.double().cpu().numpy()
    bound, lse_bound = _kv.tolerance(weight, reach, want, max(max(lengths), 1), dim, bf16)
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(lse))
    fin = np.isfinite(lse)
    assert (np.abs(got_lse[fin] - lse[fin]) <= (lse_bound + 2.0 ** -23 * np.abs(lse))[fin]).all()
    off = np.abs(got - want) / bound
    assert np.isfinite(off).all()
    at = np.unravel_index(off.argmax(), off.shape)
    assert off.max() <= 1, f"{off.max()} of the bound at {at}: {got[at]} for {want[at]}"
    return got


CASES = [
    # kv heads, group, block, dim, dtype, new, before
    (1, 1, 16, 64, "bf16", [1], [0]),
    (2, 4, 16, 128, "bf16", [1], [15]),
    (2, 8, 64, 128, "bf16", [1, 1, 1, 1, 1], [0, 62, 63, 64, 700]),
    (3, 5, 32, 64, "bf16", [1, 0, 2], [31, 40, 333]),
    (1, 7, 128, 192, "bf16", [2, 1], [126, 511]),
    (2, 16, 32, 256, "bf16", [1, 1], [1, 1000]),
    (1, 17, 16, 64, "bf16", [1, 3], [77, 5]),
    (1, 40, 64, 128, "bf16", [1, 2], [130, 64]),
    (4, 1, 256, 128, "bf16", [5, 1, 3], [300, 255, 0]),
    (2, 2, 16, 64, "fp32", [1, 2, 1], [0, 100, 517]),
    (1, 6, 64, 128, "fp32", [1, 3], [1000, 60]),
    (2, 1, 32, 256, "fp32", [4, 1], [33, 2]),
    (1, 3, 16, 192, "fp32", [1], [64]),
    # chunks and prompts
    (2, 2, 16, 64, "bf16", [33, 1, 64], [0, 50, 17]),
    (1, 8, 64, 128, "bf16", [130, 100], [0, 333]),
    (2, 3, 32, 128, "bf16", [47, 65], [64, 1]),
    (1, 4, 128, 256, "bf16", [70], [200]),
    (1, 5, 64, 192, "bf16", [129], [63]),
    (1, 20, 32, 64, "bf16", [40, 40], [3, 40]),
    (1, 2, 16, 128, "fp32", [66, 40], [30, 0]),
    (2, 1, 64, 64, "fp32", [130], [70]),
]


@pytest.mark.parametrize("heads,group,block,dim,dtype,new,before", CASES)
def test_causal(heads, group, block, dim, dtype, new, before):
    announce(f"kv attention {heads}x{group} heads, pages of {block} x {dim}, {dtype}, "
             f"{new} after {before}")
    ref, cu, lengths, table = filled(new, before, heads, block, dim)
    q = queries(cu[-1], heads * group, dim, dtype, 1)
    check(ref, ref.device(fp4), q, cu, lengths, table)


@pytest.mark.parametrize("heads,group,block,dim,dtype,new,before", CASES[2:4] + CASES[9:11] + CASES[13:15] + CASES[19:20])
@pytest.mark.parametrize("window", [1, 15, 64, 100])
def test_window(heads, group, block, dim, dtype, new, before, window):
    announce(f"kv attention, window {window}, {heads}x{group}, {block} x {dim}, {dtype}, {new} "
             f"after {before}")
    ref, cu, lengths, table = filled(new, before, heads, block, dim)
    q = queries(cu[-1], heads * group, dim, dtype, 2)
    check(ref, ref.device(fp4), q, cu, lengths, table, window=window)


@pytest.mark.parametrize("heads,group,block,dim,dtype,new,before", CASES[2:4] + CASES[9:11] + CASES[13:15])
def test_not_causal(heads, group, block, dim, dtype, new, before):
    announce(f"kv attention, not causal, {heads}x{group}, {block} x {dim}, {dtype}, {new} after "
             f"{before}")
    ref, cu, lengths, table = filled(new, before, heads, block, dim)
    q = queries(cu[-1], heads * group, dim, dtype, 3)
    check(ref, ref.device(fp4), q, cu, lengths, table, causal=False)


@pytest.mark.parametrize("length", [1, 2, 31, 32, 33, 255, 256, 257, 511, 513, 1023, 1025, 4097])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_lengths_of_one_token(length, dtype):
    """A single token after any number of others, one conversation: the split
    over the keys and its joints."""
    announce(f"kv attention of one token at length {length}, {dtype}")
    ref, cu, lengths, table = filled([1], [length - 1], 1, 16, 64, seed=length)
    q = queries(1, 4, 64, dtype, 4)
    check(ref, ref.device(fp4), q, cu, lengths, table)


def test_scales():
    """Scores scaled by more than usual, negatively, and by zero."""
    ref, cu, lengths, table = filled([2, 1], [100, 500], 2, 32, 128)
    q = queries(3, 8, 128, "bf16", 5)
    for scale in (0.0, -0.07, 3.0):
        announce(f"kv attention, scale {scale}")
        check(ref, ref.device(fp4), q, cu, lengths, table, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new", [1, 40])
def test_rows_that_see_nothing(new, dtype):
    """Sequences without tokens, positions before 0, and rows of no sequence."""
    ref, cu, lengths, table = filled([new, new, new], [0, 3, 70], 2, 16, 64)
    q = queries(cu[-1] + 5, 6, 64, dtype, 6)
    dev = ref.device(fp4)
    lengths = [0, new // 2, new + 70]  # the first sees nothing, half of the second neither
    announce(f"kv attention, rows that see nothing, {new} new, {dtype}")
    got, lse = fp4.kv_attention(q.cuda(), dev, *_kv.batch(fp4, cu, lengths, table),
                                return_lse=True)
    empty = list(range(new)) + list(range(new, 2 * new - new // 2)) + list(range(cu[-1], cu[-1] + 5))
    assert bool((got[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())
    rest = [t for t in range(cu[-1]) if t not in empty]
    assert bool((got[rest] != 0).any(-1).all()) and bool(lse[rest].isfinite().all())
    full = _kv.attention(ref, q.double().numpy()[2 * new:cu[-1]], [0, 0, 0, new], [0, 0, new + 70],
                         table, 64 ** -0.5)
    bound, _ = _kv.tolerance(full[2], full[3], full[0], new + 70, 64, dtype == "bf16")
    assert (np.abs(got[2 * new:cu[-1]].double().cpu().numpy() - full[0]) <= bound).all()


@pytest.mark.parametrize("new", [1, 50])
def test_nan_is_seen_by_its_rows_only(new):
    """A NaN key or value reaches the rows that see it, and no other; NaN codes
    and scales past a sequence's end reach none."""
    heads, block, dim = 2, 32, 64
    ref, cu, lengths, table = filled([new, new], [90, 90], heads, block, dim)
    where = 90 + new // 2
    ref.codes[0][table[0][where // block], 0, where % block, 5] = 127
    ref.codes[1][table[1][where // block], 1, where % block, 6] = 255
    q = queries(2 * new, 2 * heads, dim, "bf16", 7)
    announce(f"kv attention over NaN, {new} new")
    got = fp4.kv_attention(q.cuda(), ref.device(fp4), *_kv.batch(fp4, cu, lengths, table))
    nan = got.isnan().cpu()
    want = torch.zeros_like(nan)
    want[new // 2:new, :2] = True          # a NaN score takes its whole row
    want[new + new // 2:, 2:, 6] = True    # a NaN value takes its own dimension
    assert torch.equal(nan, want)


def test_extreme_scales():
    """Values near the lower end of the fp32 range: their sums are subnormal."""
    ref, cu, lengths, table = filled([1], [40], 1, 16, 64)
    ref.scales[1][:] = 3  # values near 2^-124
    q = queries(1, 2, 64, "fp32", 8)
    announce("kv attention with tiny values")
    got = fp4.kv_attention(q.cuda(), ref.device(fp4), *_kv.batch(fp4, cu, lengths, table))
    want, _, weight, reach = _kv.attention(ref, q.double().numpy(), cu, lengths, table, 0.125)
    # fp32 subnormal sums: a step of 2^-149 a key
    bound, _ = _kv.tolerance(weight, reach, want, 41, 64, False)
    assert (np.abs(got.double().cpu().numpy() - want) <= bound + 41 * 2.0 ** -126).all()


@pytest.mark.parametrize("new,dtype", [(1, "bf16"), (1, "fp32"), (40, "bf16")])
@pytest.mark.parametrize("apart", [1, 12, 21])
def test_pages_of_far_apart_scales(new, dtype, apart):
    """Values 2^-apart of another page's, which nothing weighs: as exact as ever."""
    cu, lengths, table, pages = _kv.layout([new], [32], 16)
    ref = _kv.Cache(pages, 1, 16, 64)
    g = np.random.default_rng(0)
    k, v = (g.standard_normal((32 + new, 1, 64)) for _ in range(2))
    k[:16, :, 0], k[16:, :, 0] = -25, 25
    v[16:] *= 2.0 ** -apart
    ref.write((k, v), [0, 32 + new], [32 + new], table)
    q = queries(new, 4, 64, dtype, 12) * 0.25
    q[:, :, 0] = 12
    announce(f"kv attention, pages 2^-{apart} apart, {new} new, {dtype}")
    # the large page's probabilities are below 2^-100: not a part of any bound
    check(ref, ref.device(fp4), q, cu, lengths, table)


@pytest.mark.parametrize("new", [1, 40])
def test_keys_out_of_bounds(new):
    """A page id the cache does not have: flagged, its keys are not seen."""
    ref, cu, lengths, table = filled([new, new], [64, 80], 1, 16, 64)
    q = queries(2 * new, 2, 64, "bf16", 9)
    dev = ref.device(fp4)
    bad = [r[:] for r in table]
    bad[0][1] = ref.codes[0].shape[0]
    announce(f"kv attention, a page out of bounds, {new} new")
    args = _kv.batch(fp4, cu, lengths, bad)
    with pytest.raises(ValueError, match="out of bounds"):
        fp4.kv_attention(q.cuda(), dev, *args)
    got = fp4.kv_attention(q.cuda(), dev, *args, check=False)
    good = fp4.kv_attention(q.cuda(), dev, *_kv.batch(fp4, cu, lengths, table))
    assert torch.equal(got[new:], good[new:])
    # without positions 16 .. 31: the same pages in a table that lacks that one
    # are a sequence 16 shorter, every row at its own end
    cut = [bad[0][:1] + bad[0][2:] + [0], bad[1]]
    less = fp4.kv_attention(q.cuda(), dev, *_kv.batch(fp4, cu, [lengths[0] - 16, lengths[1]], cut))
    torch.testing.assert_close(got[:new].float(), less[:new].float(), rtol=2.0 ** -6, atol=2.0 ** -8)


def test_strided_queries_and_stream():
    """Queries that are slices of a fused projection's rows, on a side stream."""
    ref, cu, lengths, table = filled([1, 30], [50, 70], 2, 32, 128)
    q = queries(31, 8, 128, "bf16", 10)
    dev = ref.device(fp4)
    args = _kv.batch(fp4, cu, lengths, table)
    want = fp4.kv_attention(q.cuda(), dev, *args)
    fused = torch.randn(31, 12 * 128, device="cuda").bfloat16()
    part = fused.view(31, 12, 128)[:, 2:10]
    part.copy_(q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    announce("kv attention of strided queries on a side stream")
    with torch.cuda.stream(stream):
        got = fp4.kv_attention(part, dev, *args)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(got, want)


def test_same_result_every_time():
    ref, cu, lengths, table = filled([1, 1], [3000, 500], 2, 16, 64)
    q = queries(2, 8, 64, "bf16", 11).cuda()
    dev, args = ref.device(fp4), _kv.batch(fp4, cu, lengths, table)
    announce("kv attention, ten times the same")
    first = fp4.kv_attention(q, dev, *args, return_lse=True)
    for _ in range(9):
        again = fp4.kv_attention(q, dev, *args, return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_offsets_past_32_bits():
    heads, block, dim, pages = 8, 64, 128, (1 << 32) // (8 * 64 * 128) + 40
    dev = fp4.new_kv_cache(pages, heads, block, dim, "cuda")
    far, near = [pages - 1, pages - 9, pages - 30], [4, 2, 9]
    x = torch.randn(150, heads, dim, device="cuda")
    q = torch.randn(1, 2 * heads, dim, device="cuda").bfloat16()
    announce("kv attention past 2^32 bytes")
    outs = []
    for pages_of in (far, near):
        args = _kv.batch(fp4, [0, 150], [150], [pages_of])
        fp4.kv_cache_write(dev, x, x, *args)
        outs.append(fp4.kv_attention(q, dev, *_kv.batch(fp4, [0, 1], [150], [pages_of])))
    assert torch.equal(*outs)


def test_graph_replays():
    """Write and attention captured once and replayed with other inputs in the
    same buffers, eager work between the replays."""
    block, heads, dim = 16, 2, 64
    ref, cu, lengths, table = filled([1, 1, 1], [20, 300, 45], heads, block, dim)
    dev, args = ref.device(fp4), _kv.batch(fp4, cu, lengths, table)
    same = fp4.KVCache(*(t.clone() for t in (dev.k_codes, dev.k_scales, dev.v_codes, dev.v_scales)))
    k, v = (torch.randn(3, heads, dim, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(3, 4 * heads, dim, device="cuda").bfloat16()

    def step(cache):
        fp4.kv_cache_write(cache, k, v, *args, check=False)
        return fp4.kv_attention(q, cache, *args, check=False)

    announce("kv write and attention in a graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(dev)
    torch.cuda.current_stream().wait_stream(side)
    step(same)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(dev)
    for i in range(4):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, device="cuda") * (i + 1))
        graph.replay()
        want = step(same)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert torch.equal(dev.k_codes, same.k_codes) and torch.equal(dev.v_scales, same.v_scales)


def test_refusals():
    dev = fp4.new_kv_cache(4, 2, 16, 64, "cuda")
    args = _kv.batch(fp4, [0, 2], [2], [[1]])
    q = torch.zeros(2, 4, 64, device="cuda").bfloat16()
    for bad in (q[:, :3], q[..., :32], q.cpu()):
        with pytest.raises((ValueError, fp4.Fp4Error)):
            fp4.kv_attention(bad, dev, *args)
    with pytest.raises(TypeError):
        fp4.kv_attention(q.half(), dev, *args)
    with pytest.raises(fp4.Fp4Error):
        fp4.kv_attention(q, dev, *args, window=4, causal=False)
    with pytest.raises(fp4.Fp4Error):
        fp4.kv_attention(q, dev, *args, window=-1)
    with pytest.raises(fp4.Fp4Error):
        fp4.kv_attention(q, dev, *args, scale=math.nan)
    with pytest.raises(ValueError):
        fp4.kv_attention(q, dev, *args, out=torch.zeros(2, 4, 64, device="cuda"))
    assert fp4.kv_attention(q[:0], dev, *_kv.batch(fp4, [0, 0], [2], [[1]])).shape == (0, 4, 64)
