"""GPU tests of the 8-bit key/value cache's write and read: codes, scale bytes
and read values must equal the definition in 64 bits, bit for bit."""
import math

import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _kv
from tests._gpu import announce

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rows(tokens, heads, dim, dtype, seed, std=1.0):
    """Keys or values with a few wide channels, as a slice of wider rows."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, heads + 3, dim + 8, generator=g) * std
    x[:, :, 5::32] *= 11
    return x.to(dtype)[:, 1:1 + heads, 8:]


def as64(x):
    return x.to(torch.float64).numpy()


def on_gpu(x):
    """The same slice of the same wider rows on the GPU: strides kept."""
    base = torch.empty(x.shape[0], x.stride(0), dtype=x.dtype, device="cuda")
    y = base.as_strided(x.shape, x.stride(), x.storage_offset() % x.stride(0))
    y.copy_(x)
    return y


def same_codes(got, want, what):
    """Equal bytes; any NaN code equals any other."""
    got, want = got.cpu().numpy(), np.asarray(want)
    nan = (got & 127 == 127) & (want & 127 == 127)
    bad = np.argwhere((got != want) & ~nan)
    assert not len(bad), f"{what}: {len(bad)} differ, first at {bad[0]}: " \
                         f"{got[tuple(bad[0])]} for {want[tuple(bad[0])]}"


def same_cache(dev, ref, what):
    same_codes(dev.k_codes, ref.codes[0], what + " k codes")
    same_codes(dev.v_codes, ref.codes[1], what + " v codes")
    assert np.array_equal(dev.k_scales.cpu().numpy(), ref.scales[0]), what
    assert np.array_equal(dev.v_scales.cpu().numpy(), ref.scales[1]), what


WRITES = [
    # heads, block, dim, dtype, then the sequences' new tokens, call by call
    (2, 16, 64, "bf16", [[1], [1], [1]]),
    (1, 16, 128, "fp32", [[3, 0, 17], [1, 1, 1], [0, 40, 2]]),
    (8, 64, 128, "bf16", [[63, 64, 65, 1], [1, 1, 1, 1], [2, 0, 64, 130]]),
    (3, 32, 192, "bf16", [[5, 200], [31, 1], [1, 33]]),
    (4, 128, 256, "fp32", [[129], [128], [1], [300]]),
    (2, 256, 256, "bf16", [[257, 255], [1, 1]]),
    (5, 256, 64, "bf16", [[1] * 70, [2] * 70, [0] * 69 + [9]]),
]


@pytest.mark.parametrize("heads,block,dim,dtype,calls", WRITES)
def test_write_and_read(heads, block, dim, dtype, calls):
    total = np.sum(calls, axis=0)
    _, _, table, pages = _kv.layout(total.tolist(), [0] * len(total), block)
    ref = _kv.Cache(pages, heads, block, dim)
    dev = ref.device(fp4)
    done = np.zeros_like(total)
    for i, new in enumerate(calls):
        announce(f"kv write {heads} heads, pages of {block} x {dim}, {dtype}, call {i}: {new}")
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        done += new
        # scales grow from call to call
        k = rows(cu[-1], heads, dim, TYPES[dtype], 10 * i, std=0.3 * 5.0 ** i)
        v = rows(cu[-1], heads, dim, TYPES[dtype], 10 * i + 1, std=4.0 ** -i)
        ref.write((as64(k), as64(v)), cu, done.tolist(), table)
        args = _kv.batch(fp4, cu, done.tolist(), table)
        fp4.kv_cache_write(dev, on_gpu(k), on_gpu(v), *args)
        same_cache(dev, ref, f"call {i}")
        fp4.kv_cache_write(dev, on_gpu(k), on_gpu(v), *args)  # the same again changes nothing
        same_cache(dev, ref, f"call {i} again")
        for out in (torch.float32, torch.bfloat16):
            got = fp4.kv_cache_read(dev, *args, cu[-1], out_dtype=out)
            whole = fp4.kv_cache_read(dev, _kv.batch(fp4, [0] + np.cumsum(done).tolist(), [1], [[1]])[0],
                                      *args[1:], int(done.sum()), out_dtype=out)
            for half in range(2):
                want = [ref.sequence(half, table[s], int(n)) for s, n in enumerate(done)]
                new_rows = [w[len(w) - n:] for w, n in zip(want, new)]
                assert np.array_equal(as64(got[half].cpu()), np.concatenate(new_rows))
                assert np.array_equal(as64(whole[half].cpu()), np.concatenate(want))


@pytest.mark.parametrize("value", [0.0, -0.0, 448.0, 449.0, 3.3e38, -1e-37, 1e-40, 1.4e-45, 224.0,
                                   225.0, 0.875, 0.8750001])
def test_scale_of_one_value(value):
    """Ends of the scale's range: zero, subnormals, the largest, ties at 1.75 2^e."""
    cu, lengths, table, pages = _kv.layout([1], [0], 16)
    ref = _kv.Cache(pages, 1, 16, 64)
    dev = ref.device(fp4)
    x = torch.zeros(1, 1, 64)
    x[0, 0, 7], x[0, 0, 9] = value, value / 3
    announce(f"kv write of {value}")
    ref.write((as64(x), as64(-x)), cu, lengths, table)
    fp4.kv_cache_write(dev, x.cuda(), (-x).cuda(), *_kv.batch(fp4, cu, lengths, table))
    same_cache(dev, ref, f"{value}")


def test_growth_by_every_step():
    """A page's first token at each distance below a later one."""
    steps = list(range(0, 60, 3)) + [120, 250]
    cu, lengths, table, pages = _kv.layout([1] * len(steps), [0] * len(steps), 16)
    ref = _kv.Cache(pages, 1, 16, 64)
    dev = ref.device(fp4)
    g = torch.Generator().manual_seed(3)
    small = torch.randn(len(steps), 1, 64, generator=g)
    small *= torch.tensor([2.0 ** -(s // 2) for s in steps])[:, None, None]
    large = torch.randn(len(steps), 1, 64, generator=g)
    large *= torch.tensor([2.0 ** (s - s // 2) for s in steps])[:, None, None]
    announce("kv write, growing scales")
    for i, x in enumerate((small, large)):
        ref.write((as64(x), as64(x)), cu, [i + 1] * len(steps), table)
        fp4.kv_cache_write(dev, x.cuda(), x.cuda(),
                           *_kv.batch(fp4, cu, [i + 1] * len(steps), table))
    same_cache(dev, ref, "grown")


def test_values_that_are_not_finite():
    cu, lengths, table, pages = _kv.layout([20, 3], [0, 0], 16)
    ref = _kv.Cache(pages, 2, 16, 64)
    dev = ref.device(fp4)
    x = torch.randn(23, 2, 64, generator=torch.Generator().manual_seed(1))
    x[4, 0, 3], x[17, 1, 0], x[22, 0, 63] = math.nan, math.inf, -math.inf
    ref.write((as64(x), as64(x)), cu, lengths, table)
    announce("kv write of NaN and infinities")
    args = _kv.batch(fp4, cu, lengths, table)
    with pytest.raises(ValueError, match="finite"):
        fp4.kv_cache_write(dev, x.cuda(), x.cuda(), *args)
    same_cache(dev, ref, "not finite")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp4.kv_cache_write(dev, x.cuda(), x.cuda(), *args, check=False, status=status)
    assert int(status.item()) == fp4.FLAG_NONFINITE


def test_read_every_code_and_scale():
    """All 256 codes under all 256 scale bytes, in fp32 and bf16."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1, 16, 1)  # [256, 1, 16, 256]
    scales = torch.arange(256, dtype=torch.uint8)[:, None].contiguous()
    dev = fp4.KVCache(codes.cuda(), scales.cuda(), codes.flip(3).contiguous().cuda(), scales.cuda())
    args = _kv.batch(fp4, [0, 4096], [4096], [list(range(256))])
    announce("kv read of every code and scale byte")
    want = _kv.VALUES[None, :] * np.array([_kv.scale_value(b) for b in range(256)])[:, None]
    with np.errstate(over="ignore"):
        exact = torch.from_numpy(want).to(torch.float32)  # every product is an fp32 value, or over
    for dtype in (torch.float32, torch.bfloat16):
        k, v = fp4.kv_cache_read(dev, *args, 4096, out_dtype=dtype)
        w = exact.to(dtype).float()
        for got, expect in ((k, w), (v, w.flip(1))):
            got = got.cpu().float().view(256, 16, 256)
            expect = expect[:, None, :].expand(-1, 16, -1)
            assert torch.equal(got.isnan(), expect.isnan())
            assert torch.equal(got.nan_to_num(7.0), expect.nan_to_num(7.0))


def test_rows_of_no_sequence():
    """Rows past cu[seqs] are not written, and read as zero."""
    cu, lengths, table, pages = _kv.layout([3, 18], [14, 0], 16)
    ref = _kv.Cache(pages, 2, 16, 64)
    ref.write([np.ones((17, 2, 64))] * 2, [0, 14, 14], [14, 0], table)
    dev = ref.device(fp4)
    x = torch.randn(60, 2, 64, generator=torch.Generator().manual_seed(5))
    ref.write((as64(x), as64(x)), cu, lengths, table)
    announce("kv write and read with padding rows")
    args = _kv.batch(fp4, cu, lengths, table)
    fp4.kv_cache_write(dev, x.cuda(), x.cuda(), *args)
    same_cache(dev, ref, "padded")
    k, _ = fp4.kv_cache_read(dev, *args, 60, out_dtype=torch.float32,
                             out=(torch.full((60, 2, 64), 9.0, device="cuda"),
                                  torch.full((60, 2, 64), 9.0, device="cuda")))
    assert bool((k[21:] == 0).all()) and bool((k[:21] != 9).all())


@pytest.mark.parametrize("fault", ["page", "negative page", "narrow", "before 0", "rows"])
def test_entries_out_of_bounds(fault):
    """They are flagged and skipped; the other sequence is written and read."""
    cu, lengths, table, pages = _kv.layout([20, 7], [0, 3], 16)
    ref = _kv.Cache(pages, 2, 16, 64)
    ref.write([np.ones((3, 2, 64))] * 2, [0, 0, 3], [0, 3], table)
    dev = ref.device(fp4)
    x = torch.randn(27, 2, 64, generator=torch.Generator().manual_seed(5))
    good = [r[:] for r in table]
    good_lengths, good_cu = list(lengths), list(cu)
    if fault == "page":
        table[0] = [pages] * 2
    if fault == "negative page":
        table[0] = [-1] * 2
    if fault == "narrow":
        lengths[0] = 20 + 16 * 40
    if fault == "before 0":
        lengths[0] = 0
    if fault == "rows":
        cu = [0, 60, 67]
    announce(f"kv write and read out of bounds: {fault}")
    args = _kv.batch(fp4, cu, lengths, table)
    with pytest.raises(ValueError, match="out of bounds"):
        fp4.kv_cache_write(dev, x.cuda(), x.cuda(), *args)
    if fault != "rows":
        only = as64(x)
        ref.write((only[20:], only[20:]), [0, 0, 7], [0, good_lengths[1]], good)
    same_cache(dev, ref, fault)
    with pytest.raises(ValueError, match="out of bounds"):
        fp4.kv_cache_read(dev, *args, 27)
    k, _ = fp4.kv_cache_read(dev, *args, 27, out_dtype=torch.float32, check=False,
                             out=(torch.zeros(27, 2, 64, device="cuda"),
                                  torch.zeros(27, 2, 64, device="cuda")))
    assert bool((k[:20] == 0).all())
    if fault != "rows":
        want = ref.sequence(0, good[1], good_lengths[1])[3:]
        assert np.array_equal(as64(k[good_cu[1]:].cpu()), want)


def test_offsets_past_32_bits():
    """Pages whose codes start past 2^32 bytes."""
    heads, block, dim, pages = 8, 64, 128, (1 << 32) // (8 * 64 * 128) + 40
    dev = fp4.new_kv_cache(pages, heads, block, dim, "cuda")
    table = [[pages - 1, 3, pages - 17]]
    x = rows(130, heads, dim, torch.bfloat16, 2)
    announce("kv write and read past 2^32 bytes")
    args = _kv.batch(fp4, [0, 130], [130], table)
    fp4.kv_cache_write(dev, on_gpu(x), on_gpu(x), *args)
    got, _ = fp4.kv_cache_read(dev, *args, 130, out_dtype=torch.float32)
    small = _kv.Cache(3, heads, block, dim)
    small.write((as64(x), as64(x)), [0, 130], [130], [[2, 0, 1]])
    assert np.array_equal(as64(got.cpu()), small.sequence(0, [2, 0, 1], 130))


def test_on_another_stream():
    cu, lengths, table, pages = _kv.layout([33, 5], [0, 0], 32)
    ref = _kv.Cache(pages, 2, 32, 128)
    dev = ref.device(fp4)
    x = rows(38, 2, 128, torch.bfloat16, 1)
    ref.write((as64(x), as64(x)), cu, lengths, table)
    args = _kv.batch(fp4, cu, lengths, table)
    y = on_gpu(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    announce("kv write on a side stream")
    with torch.cuda.stream(stream):
        fp4.kv_cache_write(dev, y, y, *args)
    torch.cuda.current_stream().wait_stream(stream)
    same_cache(dev, ref, "side stream")


def test_empty_batch():
    dev = fp4.new_kv_cache(4, 2, 16, 64, "cuda")
    before = dev.k_codes.clone()
    args = _kv.batch(fp4, [0, 0], [5], [[1]])
    x = torch.empty(0, 2, 64, device="cuda")
    announce("kv write and read of no rows")
    fp4.kv_cache_write(dev, x, x, *args)
    k, v = fp4.kv_cache_read(dev, *args, 0)
    assert k.shape == v.shape == (0, 2, 64) and torch.equal(before, dev.k_codes)


def test_refusals():
    dev = fp4.new_kv_cache(4, 2, 16, 64, "cuda")
    cu, lengths, table = _kv.batch(fp4, [0, 2], [2], [[1]])
    x = torch.zeros(2, 2, 64, device="cuda")
    with pytest.raises(ValueError):  # heads
        fp4.kv_cache_write(dev, x[:, :1], x[:, :1], cu, lengths, table)
    with pytest.raises(ValueError):  # k and v differ
        fp4.kv_cache_write(dev, x, x.bfloat16(), cu, lengths, table)
    with pytest.raises(TypeError):  # dtype
        fp4.kv_cache_write(dev, x.half(), x.half(), cu, lengths, table)
    with pytest.raises(TypeError):
        fp4.kv_cache_write(dev, x, x, cu.long(), lengths, table)
    with pytest.raises(ValueError):  # entries
        fp4.kv_cache_write(dev, x, x, cu[:1], lengths, table)
    with pytest.raises(ValueError):  # device
        fp4.kv_cache_write(dev, x.cpu(), x.cpu(), cu, lengths, table)
    with pytest.raises(ValueError):  # rows not dense
        t = torch.zeros(2, 2, 128, device="cuda")[..., ::2]
        fp4.kv_cache_write(dev, t, t, cu, lengths, table)
    with pytest.raises(fp4.Fp4Error):  # alignment
        t = torch.zeros(2, 2, 72, device="cuda")[..., 1:65]
        fp4.kv_cache_write(dev, t, t, cu, lengths, table)
    with pytest.raises(fp4.Fp4Error):  # page size
        odd = fp4.new_kv_cache(4, 2, 24, 64, "cuda")
        fp4.kv_cache_write(odd, x, x, cu, lengths, table)
    with pytest.raises(ValueError):  # codes and scales do not fit
        fp4.KVCache(dev.k_codes, dev.k_scales[:3], dev.v_codes, dev.v_scales)
