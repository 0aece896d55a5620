"""GPU tests of attention over the 8-bit cache where the scales of value pages
are far apart: a row's result is as exact as its own keys allow, whatever the
pages of tokens it does not see hold."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _kv, _kv_rows
from tests import test_gpu_kv_attention as plain
from tests._gpu import announce

pytestmark = pytest.mark.gpu

# new tokens, group, dim, dtype: few rows, many rows, and fp32 queries
ROWS = [(40, 4, 64, "bf16"), (40, 4, 128, "bf16"), (30, 2, 256, "bf16"), (30, 2, 192, "fp32"),
        (300, 16, 64, "bf16"), (300, 16, 128, "bf16"), (200, 20, 192, "bf16"),
        (200, 20, 256, "bf16")]


def pages_of_scales(new, before, dim, shift, seed=0):
    """One sequence whose page b has values times 2^shift(b)."""
    cu, lengths, table, pages = _kv.layout([new], [before], 16, seed=seed)
    ref = _kv.Cache(pages, 1, 16, dim, seed)
    g = np.random.default_rng(seed + 1)
    k, v = (g.standard_normal((lengths[0], 1, dim)) for _ in range(2))
    v *= np.exp2([float(shift(p // 16)) for p in range(lengths[0])])[:, None, None]
    ref.write((k, v), [0, lengths[0]], lengths, table)
    return ref, cu, lengths, table


@pytest.mark.parametrize("new,group,dim,dtype", ROWS)
@pytest.mark.parametrize("apart", [25, 45, 90])
def test_later_tokens_of_a_larger_scale(new, group, dim, dtype, apart):
    """A prompt whose first page is 2^-apart of the others: rows of the same
    tile that see only that page have its values."""
    ref, cu, lengths, table = pages_of_scales(new, 0, dim, lambda b: -apart if b == 0 else 0)
    q = plain.queries(new, group, dim, dtype, 1)
    announce(f"kv attention, later pages 2^{apart} larger, {new} x {group} rows of {dim}, {dtype}")
    batch = _kv_rows.wide_batch(fp4, cu, lengths, table)
    got, _ = _kv_rows.compare(ref, ref.device(fp4), q, cu, lengths, table, fp4=fp4, batch=batch)
    assert bool((got[:16] != 0).any(-1).all())


@pytest.mark.parametrize("new,group,dim,dtype", ROWS)
def test_scales_that_rise_and_fall(new, group, dim, dtype):
    """Page scales over 2^60, up and down."""
    ref, cu, lengths, table = pages_of_scales(new, 100, dim, lambda b: 60 - abs(60 - 7 * b % 120))
    q = plain.queries(new, group, dim, dtype, 2)
    for window in (0, 20):
        announce(f"kv attention, scales up and down, window {window}, {new} x {group} rows of {dim}, "
                 f"{dtype}")
        batch = _kv_rows.wide_batch(fp4, cu, lengths, table)
        _kv_rows.compare(ref, ref.device(fp4), q, cu, lengths, table, fp4=fp4, batch=batch,
                         window=window)


@pytest.mark.parametrize("new,group,dim,dtype", [(1, 4, 64, "bf16"), (1, 4, 256, "fp32")] + ROWS)
@pytest.mark.parametrize("apart", [30, 60, 100])
def test_scale_against_probability(new, group, dim, dtype, apart):
    """A page of values 2^apart larger whose probabilities are some 2^-108."""
    cu, lengths, table, pages = _kv.layout([new], [32], 16)
    ref = _kv.Cache(pages, 1, 16, dim)
    g = np.random.default_rng(0)
    k, v = (g.standard_normal((32 + new, 1, dim)) for _ in range(2))
    k[:16, :, 0], k[16:, :, 0] = -25, 25
    v[16:] *= 2.0 ** -apart
    ref.write((k, v), [0, 32 + new], [32 + new], table)
    q = plain.queries(new, group, dim, dtype, 12) * 0.25
    q[:, :, 0] = 12
    announce(f"kv attention, a page 2^{apart} larger that weighs little, {new} x {group} rows of "
             f"{dim}, {dtype}")
    batch = _kv_rows.wide_batch(fp4, cu, lengths, table)
    _kv_rows.compare(ref, ref.device(fp4), q, cu, lengths, table, scale=0.125, fp4=fp4, batch=batch)


@pytest.mark.parametrize("group,dim,dtype", [(4, 64, "bf16"), (16, 128, "bf16"), (20, 192, "bf16"),
                                             (4, 128, "fp32")])
def test_many_small_probabilities(group, dim, dtype):
    """One key of large probability and small values, many others of
    probabilities below fp16's range and values 2^21 larger: these decide."""
    new, before = 100, 900
    ref, cu, lengths, table = pages_of_scales(new, before, dim, lambda b: 0)
    for b, page in enumerate(table[0][:-(-lengths[0] // 16)]):
        ref.codes[0][page, :, :, 0] = _kv.e4m3_codes(np.array(8.0 if b == 0 else 0.0))
        ref.scales[0][page], ref.scales[1][page] = 127, 106 if b == 0 else 127
        ref.codes[0][page, :, :, 1:] = 0
    q = torch.zeros(new, group, dim).to(plain.TYPES[dtype])
    q[:, :, 0] = 23.0  # the first page's scores are 184 x 0.125 = 23 over the others'
    announce(f"kv attention, small probabilities of large values, {group} heads of {dim}, {dtype}")
    batch = _kv_rows.wide_batch(fp4, cu, lengths, table)
    _kv_rows.compare(ref, ref.device(fp4), q, cu, lengths, table, scale=0.125, fp4=fp4, batch=batch)
