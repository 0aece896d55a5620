"""The norm and rotation of queries and keys, against 64 bits."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests._gpu import announce

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def frequencies(rotary, base=10000.0):
    return base ** -(torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)


def reference(x, weight, pos, freq, eps, interleaved):
    """y in float64, and what its error is relative to: the pair's length."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    angle = pos.double()[:, None, None] * freq
    c, s = torch.cos(angle), torch.sin(angle)
    r = 2 * freq.numel()
    first, second = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2),
                                                                          slice(r // 2, r))
    y, size = x.clone(), x.abs()
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    size[..., first] = size[..., second] = torch.hypot(a, b)
    return y, size


def batch_of(new, old):
    cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32)
    lengths = torch.tensor([n + o for n, o in zip(new, old)], dtype=torch.int32)
    pos = torch.cat([torch.arange(o, o + n) for n, o in zip(new, old)])
    return cu, lengths, pos


def check(got, want, size, dtype, far=0.0):
    got = got.cpu()
    assert got.dtype == dtype and not got.isnan().any()
    # the norm: 256 squares added in five steps or more, root, quotient and two
    # products; cosine and sine rounded, two products added: fewer than 2^5 roundings
    bound = (2.0 ** -19 + far) * size + torch.finfo(dtype).eps / 2 * 1.01 * want.abs() + 1e-37
    err = (got.double() - want).abs()
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary,heads,kv,weights,new,old", [
    (64, 64, 8, 2, "both", [1], [0]), (64, 32, 5, 5, None, [3, 0, 9], [10, 4, 0]),
    (128, 128, 64, 8, "both", [1, 1, 1], [999, 0, 70000]), (128, 64, 7, 1, "q", [130], [5]),
    (128, 16, 1, 1, "k", [2, 5], [0, 1]), (192, 192, 3, 1, "both", [4, 1], [77, 3]),
    (192, 96, 12, 4, "both", [65], [0]), (256, 256, 16, 2, "both", [1, 7], [2, 2 ** 20]),
    (256, 128, 9, 3, None, [40], [100]), (128, 128, 40, 8, "both", [700, 400], [0, 3000]),
    (128, 112, 40, 8, "both", [1] * 130, range(130))])
def test_rows(dim, rotary, heads, kv, weights, new, old, interleaved, dtype):
    announce(f"norm_rotate {dim} {rotary} {heads} {kv} {weights} {dtype} {interleaved}")
    dtype = DTYPES[dtype]
    g = torch.Generator().manual_seed(dim + rotary + heads)
    cu, lengths, pos = batch_of(new, old)
    x = torch.randn(len(pos), heads + 2 * kv, dim, generator=g)
    x = (x * torch.exp2(torch.randint(-6, 7, (len(pos), heads + 2 * kv, 1), generator=g))).to(dtype)
    w = (1 + 0.5 * torch.randn(2, dim, generator=g)).to(dtype)
    qw = w[0].contiguous() if weights in ("both", "q") else None
    kw = w[1].contiguous() if weights in ("both", "k") else None
    freq = frequencies(rotary)
    xd = x.cuda()  # q, k, v as one projection gives them
    dev = lambda t: None if t is None else t.cuda()
    q, k = fp4.norm_rotate(xd[:, :heads], xd[:, heads:heads + kv], cu.cuda(), lengths.cuda(),
                           freq.cuda(), dev(qw), dev(kw), eps=1e-5, interleaved=interleaved)
    assert q.is_contiguous() and k.is_contiguous()
    for got, rows, weight in ((q, x[:, :heads], qw), (k, x[:, heads:heads + kv], kw)):
        check(got, *reference(rows, weight, pos, freq, 1e-5, interleaved), dtype)
    # in place, with fp32 weights where they are bf16
    f32 = lambda t: None if t is None else t.float().cuda()
    slices = xd[:, :heads], xd[:, heads:heads + kv]
    fp4.norm_rotate(*slices, cu.cuda(), lengths.cuda(), freq.cuda(), f32(qw), f32(kw), eps=1e-5,
                    interleaved=interleaved, out=slices)
    assert torch.equal(slices[0], q) and torch.equal(slices[1], k)
    assert torch.equal(xd[:, heads + kv:].cpu(), x[:, heads + kv:])


@pytest.mark.parametrize("pos", [2 ** 24 + 1, 2 ** 27 - 1, 2 ** 31 - 8])
def test_far_positions(pos):
    """Angles of 2^31 radians, still in fp32's precision."""
    freq = torch.tensor([1.0, 0.9, 1 / 3, 1e-3, 2e-9, 0.0, 3.0, 0.5], dtype=torch.float64)
    cu, lengths, at = batch_of([7], [pos])
    g = torch.Generator().manual_seed(1)
    x = torch.randn(7, 2, 64, generator=g)
    q, k = fp4.norm_rotate(x.cuda(), x[:, :1].cuda().contiguous(), cu.cuda(), lengths.cuda(),
                           freq.cuda())
    # the reference's own angle is rounded to 2^-53 of itself
    far = float(at.max()) * 3 * 2.0 ** -52
    want, size = reference(x, None, at, freq, 0, False)
    check(q, want, size, torch.float32, far)
    check(k, want[:, :1], size[:, :1], torch.float32, far)


def test_rows_of_no_sequence_and_bad_batches():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(9, 3, 64, generator=g).cuda()
    freq = frequencies(64).cuda()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    # two rows behind the last sequence, one sequence without new tokens
    q, k = fp4.norm_rotate(x, x, i32(0, 4, 4, 7), i32(10, 3, 7), freq)
    whole, _ = fp4.norm_rotate(x[:7], x[:7], i32(0, 4, 4, 7), i32(10, 3, 7), freq)
    assert torch.equal(q[:7], whole) and (q[7:] == 0).all() and (k[7:] == 0).all()
    status = i32(0)
    for cu, lengths in (((0, 4, 9), (3, 5)),        # a position of -1
                        ((1, 4, 9), (9, 9)), ((0, 12, 9), (9, 9)), ((0, 4, 20), (9, 20)),
                        ((0, -4, 9), (9, 9))):
        status.zero_()
        q, _ = fp4.norm_rotate(x, x, i32(*cu), i32(*lengths), freq, check=False, status=status)
        assert status.item() == fp4.FLAG_CACHE_INDEX, (cu, lengths)
        with pytest.raises(ValueError):
            fp4.norm_rotate(x, x, i32(*cu), i32(*lengths), freq)
    q, _ = fp4.norm_rotate(x, x, i32(0, 4, 9), i32(3, 5), freq, check=False)
    assert (q[0] == 0).all() and (q[1] == x[1]).all()  # position 0 turns nothing
    assert fp4.norm_rotate(x[:0], x[:0], i32(0, 0), i32(5), freq)[0].shape == (0, 3, 64)


def test_values_that_are_not_finite():
    x = torch.ones(4, 2, 128)
    x[1, 0, 100], x[2, 1, 3] = float("nan"), float("inf")
    w = torch.ones(128)
    cu, lengths, pos = batch_of([4], [0])
    q, _ = fp4.norm_rotate(x.cuda(), x.cuda(), cu.cuda(), lengths.cuda(), frequencies(128).cuda(),
                           w.cuda(), w.cuda())
    q = q.cpu()
    assert q[1, 0].isnan().all() and q[2, 1].isnan().any()
    q[1, 0], q[2, 1] = 0, 0
    assert q.isfinite().all()
    # zeros stay zeros, whatever eps adds to them
    q, _ = fp4.norm_rotate(0 * torch.ones(1, 1, 64).cuda(), torch.ones(1, 1, 64).cuda(),
                           *(t.cuda() for t in batch_of([1], [3])[:2]), frequencies(64).cuda(),
                           torch.ones(64).cuda())
    assert (q == 0).all()


def test_many_sequences():
    """More sequences than one step of the search sees."""
    n = 5000
    new = (torch.arange(n) % 3).tolist()
    old = (torch.arange(n) * 7 % 1000).tolist()
    cu, lengths, pos = batch_of(new, old)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(len(pos), 1, 64, generator=g)
    freq = frequencies(64)
    q, k = fp4.norm_rotate(x.cuda(), x.cuda(), cu.cuda(), lengths.cuda(), freq.cuda())
    want, size = reference(x, None, pos, freq, 0, False)
    check(q, want, size, torch.float32)
    assert torch.equal(q, k)


def test_captured():
    freq = frequencies(128).cuda()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 6, 128, device="cuda").bfloat16()
    w = torch.ones(128, device="cuda")
    graph = torch.cuda.CUDAGraph()
    fp4.norm_rotate(x, x, cu, lengths, freq, w, w, check=False)
    with torch.cuda.graph(graph):
        q, _ = fp4.norm_rotate(x, x, cu, lengths, freq, w, w, check=False)
    for _ in range(4):
        lengths += 1
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, fp4.norm_rotate(x, x, cu, lengths, freq, w, w)[0])
