"""GPU tests of attention over the 8-bit key/value cache where many rows share
a tile: the cases of tests/test_gpu_kv_attention.py with tables far wider than
the sequences are long, for which the work is laid out as for long ones, and
batches of more sequences than a wave has lanes."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _kv
from tests import test_gpu_kv_attention as plain
from tests._gpu import announce

pytestmark = pytest.mark.gpu


@pytest.fixture
def wide_tables(monkeypatch):
    """Tables of 2^16 pages, the rest of them ids no cache has."""
    batch = _kv.batch

    def wide(fp4, cu, lengths, table):
        cu, lengths, table = batch(fp4, cu, lengths, table)
        return cu, lengths, torch.nn.functional.pad(table, (0, 2 ** 16 - table.shape[1]),
                                                    value=2 ** 30)
    monkeypatch.setattr(_kv, "batch", wide)


CASES = [
    # kv heads, group, block, dim, dtype, new, before
    (2, 4, 16, 64, "bf16", [33, 1, 164], [0, 50, 17]),
    (1, 20, 32, 64, "bf16", [40, 40], [3, 40]),
    (1, 8, 64, 128, "bf16", [130, 100], [0, 333]),
    (2, 3, 32, 128, "bf16", [47, 65], [64, 1]),
    (1, 1, 256, 128, "bf16", [2100], [90]),
    (1, 5, 64, 192, "bf16", [129], [63]),
    (1, 4, 128, 256, "bf16", [70], [200]),
    (4, 1, 16, 256, "bf16", [100, 0, 260], [31, 40, 0]),
]


@pytest.mark.parametrize("heads,group,block,dim,dtype,new,before", CASES)
def test_causal(wide_tables, heads, group, block, dim, dtype, new, before):
    plain.test_causal(heads, group, block, dim, dtype, new, before)


@pytest.mark.parametrize("heads,group,block,dim,dtype,new,before", CASES[:4] + CASES[5:])
@pytest.mark.parametrize("window", [1, 15, 64, 100])
def test_window(wide_tables, heads, group, block, dim, dtype, new, before, window):
    plain.test_window(heads, group, block, dim, dtype, new, before, window)


@pytest.mark.parametrize("heads,group,block,dim,dtype,new,before", CASES[:4] + CASES[5:])
def test_not_causal(wide_tables, heads, group, block, dim, dtype, new, before):
    plain.test_not_causal(heads, group, block, dim, dtype, new, before)


def test_scales(wide_tables):
    ref, cu, lengths, table = plain.filled([40], [500], 2, 32, 128)
    q = plain.queries(40, 8, 128, "bf16", 5)
    for scale in (0.0, -0.07, 3.0):
        announce(f"kv attention of 40 tokens, scale {scale}")
        plain.check(ref, ref.device(fp4), q, cu, lengths, table, scale=scale)


def test_rows_that_see_nothing(wide_tables):
    plain.test_rows_that_see_nothing(60, "bf16")


def test_nan_is_seen_by_its_rows_only(wide_tables):
    plain.test_nan_is_seen_by_its_rows_only(100)


@pytest.mark.parametrize("apart", [1, 12, 21])
def test_pages_of_far_apart_scales(wide_tables, apart):
    plain.test_pages_of_far_apart_scales(40, "bf16", apart)


def test_keys_out_of_bounds(wide_tables):
    plain.test_keys_out_of_bounds(100)


def test_split_keys():
    """A chunk over a long sequence, its keys split over workgroups."""
    ref, cu, lengths, table = plain.filled([100], [8911], 3, 32, 64)
    q = plain.queries(100, 12, 64, "bf16", 1)
    announce("kv attention of 100 tokens over 9011 keys")
    plain.check(ref, ref.device(fp4), q, cu, lengths, table)


@pytest.mark.parametrize("dim,before", [(64, 70), (128, 0)])
def test_many_rows(dim, before):
    """131072 rows and more: heads are compared that start, end and cross a
    tile of 256."""
    new, group = 517, 255
    ref, cu, lengths, table = plain.filled([new], [before], 1, 64, dim)
    q = plain.queries(new, group, dim, "bf16", 2)
    announce(f"kv attention of {new} tokens, {group} heads of {dim}")
    got = fp4.kv_attention(q.cuda(), ref.device(fp4), *_kv.batch(fp4, cu, lengths, table))
    some = [0, 1, 100, 253, 254]
    want, _, weight, reach = _kv.attention(ref, q.double().numpy()[:, some], cu, lengths, table,
                                           dim ** -0.5)
    bound, _ = _kv.tolerance(weight, reach, want, new + before, dim, True)
    assert (np.abs(got[:, some].double().cpu().numpy() - want) <= bound).all()


def many(seqs, top=8):
    """Row counts of 0 to top - 1 and lengths before them."""
    g = np.random.default_rng(seqs)
    new, before = g.integers(0, top, seqs).tolist(), g.integers(0, 40, seqs).tolist()
    new[0] = new[-1] = 0
    return new, before


@pytest.mark.parametrize("seqs", [62, 63, 64, 65, 128, 254, 255, 256, 300])
def test_many_sequences(seqs):
    """A tile's place in the batch."""
    ref, cu, lengths, table = plain.filled(*many(seqs), 1, 16, 64)
    q = plain.queries(cu[-1], 3, 64, "fp32", 3)
    announce(f"kv attention of {seqs} sequences")
    plain.check(ref, ref.device(fp4), q, cu, lengths, table)


@pytest.mark.parametrize("seqs,top", [(63, 8), (65, 8), (255, 8), (256, 8), (300, 8), (65, 300),
                                      (255, 200), (256, 200)])
def test_values_name_their_sequence(seqs, top):
    """Values that are digits of their sequence's number: every row has its
    own's, exactly."""
    new, before = many(seqs, top)
    ref, cu, lengths, table = plain.filled(new, before, 2, 16, 64)
    digit = _kv.e4m3_codes(np.arange(1, 17, dtype=np.float64))
    want = np.zeros((cu[-1], 6, 64))
    for s, pages in enumerate(table):
        own = (s >> (4 * (np.arange(64) % 3))) & 15
        for page in pages[:-(-lengths[s] // 16)]:
            ref.codes[1][page] = digit[own]
            ref.scales[1][page] = 127
        want[cu[s]:cu[s + 1]] = own + 1
    q = plain.queries(cu[-1], 6, 64, "bf16", 3)
    announce(f"kv attention of {seqs} sequences of up to {top} tokens, values that name them")
    got = fp4.kv_attention(q.cuda(), ref.device(fp4), *_kv.batch(fp4, cu, lengths, table))
    assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("new", [3, 40])
def test_rows_out_of_order(new):
    """Row counts that are no prefix sum: flagged, other sequences as ever."""
    ref, cu, lengths, table = plain.filled([new] * 3, [20, 30, 40], 1, 16, 64)
    q = plain.queries(cu[-1], 2, 64, "bf16", 5).cuda()
    dev = ref.device(fp4)
    announce(f"kv attention, rows out of order, {new} new")
    want = fp4.kv_attention(q, dev, *_kv.batch(fp4, cu, lengths, table))
    for bad in ([0, new, -5, 3 * new], [0, new, 3 * new + 1, 3 * new], [0, new, 2 ** 31 - 1, 3 * new]):
        args = _kv.batch(fp4, bad, lengths, table)
        with pytest.raises(ValueError, match="out of bounds"):
            fp4.kv_attention(q, dev, *args)
        got = fp4.kv_attention(q, dev, *args, check=False)
        assert torch.equal(got[:new], want[:new])
