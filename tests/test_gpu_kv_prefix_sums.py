"""GPU tests of the cache calls' row counts and positions: prefix sums that are
none are flagged by every call, wherever in the batch they are, and entries that
do not exist read as zero over whatever the outputs held."""
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _kv
from tests._gpu import announce

pytestmark = pytest.mark.gpu


def call(what, rows, seqs, cu, lengths, table, device):
    """One call over a cache of small pages; its flags."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.ones(rows, 1, 64, device="cuda")
    batch = _kv.batch(fp4, cu, lengths, table)
    if what == "write":
        fp4.kv_cache_write(device, x, x, *batch, check=False, status=status)
    elif what == "read":
        fp4.kv_cache_read(device, *batch, rows, check=False, status=status)
    else:
        dtype = torch.bfloat16 if what == "attend bf16" else torch.float32
        q = torch.ones(rows, 12, 64, device="cuda", dtype=dtype)
        fp4.kv_attention(q, device, *batch, check=False, status=status)
    return int(status.item())


@pytest.mark.parametrize("what", ["write", "read", "attend bf16", "attend fp32"])
@pytest.mark.parametrize("seqs,new", [(1, 1), (1, 40), (3, 1), (3, 20), (62, 1), (63, 1), (64, 1),
                                      (65, 3), (255, 1), (256, 1), (256, 3), (300, 20), (5000, 1),
                                      (5000, 3)])
def test_prefix_sums(what, seqs, new):
    width = 1 + (new + 2) // 16
    lengths, table = [new + 3] * seqs, [[s * width + b for b in range(width)] for s in range(seqs)]
    good, rows = [new * s for s in range(seqs + 1)], new * seqs
    device = fp4.new_kv_cache(seqs * width, 1, 16, 64, "cuda")
    for scales in (device.k_scales, device.v_scales):
        scales.fill_(127)
    announce(f"kv {what} of {seqs} x {new} rows, prefix sums that are none")

    def flags(cu, rows=rows):
        return call(what, rows, seqs, cu, lengths, table, device) & fp4.FLAG_CACHE_INDEX

    assert not flags(good) and not flags(good, rows + 7)  # rows of no sequence are none's
    assert not flags([0] * (seqs + 1))
    assert flags([1] + good[1:])           # the first row belongs to none
    assert flags(good[:-1] + [rows + 1])   # more rows than there are
    for at in {s for s in (1, seqs // 2, seqs - 1) if 0 < s < seqs}:
        for value in (-1, good[at - 1] - 1, good[at + 1] + 1, 2 ** 31 - 1, -2 ** 31):
            assert flags(good[:at] + [value] + good[at + 1:]), (at, value)


@pytest.mark.parametrize("fault", ["page", "negative page", "narrow", "before 0"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_entries_that_do_not_exist_read_as_zero(fault, dtype):
    """Keys and values both, over outputs that held something else."""
    cu, lengths, table, pages = _kv.layout([20, 7], [0, 3], 16)
    dev = fp4.new_kv_cache(pages, 2, 16, 64, "cuda")
    x = torch.randn(30, 2, 64, generator=torch.Generator().manual_seed(5)).cuda()
    fp4.kv_cache_write(dev, x, x, *_kv.batch(fp4, [0, 20, 30], [20, 10], table))
    rows = range(20)
    if fault == "page":
        table[0] = [pages] * 2
    if fault == "negative page":
        table[0] = [table[0][0], -1]
        rows = range(16, 20)
    if fault == "narrow":
        lengths[0] = 20 + 16 * 40
    if fault == "before 0":
        lengths[0] = 8
        rows = range(12)
    announce(f"kv read of entries that do not exist: {fault}")
    out = tuple(torch.full((27, 2, 64), 9.0, device="cuda", dtype=dtype) for _ in range(2))
    fp4.kv_cache_read(dev, *_kv.batch(fp4, cu, lengths, table), 27, out=out, check=False)
    for t in out:
        zero = (t == 0).flatten(1).all(1).cpu()
        assert zero.tolist() == [i in rows for i in range(27)]
        assert not bool((t == 9).any())
