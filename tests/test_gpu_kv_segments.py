"""GPU tests of attention where one workgroup walks more than 2048 keys, whose
pages it looks up 2048 at a time: tiles of 128 and 256 rows, value scales that
rise and fall from one such segment to the next, windows, rows that see all, NaN
values and missing pages in a later segment."""
import numpy as np
import pytest

import mxfp4_block_amax_amd as fp4
from tests import _kv, _kv_rows
from tests import test_gpu_kv_attention as plain
from tests._gpu import announce

pytestmark = pytest.mark.gpu

# new tokens, query heads, dim, block: enough tiles for one workgroup of 128 (of
# the last two 256) rows each, its keys unsplit
TILES = [(513, 128, 64, 16), (513, 128, 128, 64), (258, 128, 192, 64), (258, 128, 256, 32),
         (517, 255, 64, 64), (517, 255, 128, 16)]


def segments(new, heads, dim, block, shifts, seed=0):
    """A sequence of 4200 tokens before the new ones; page scales of values
    raised by shifts[segment]."""
    ref, cu, lengths, table = plain.filled([new], [4200], 1, block, dim, seed=seed)
    for b in range(-(-lengths[0] // block)):
        ref.scales[1][table[0][b]] += np.uint8(shifts[b * block // 2048])
    q = plain.queries(new, heads, dim, "bf16", 5)
    some = [0, heads // 2 - 1, heads - 1]  # first, middle and last rows of tiles
    return ref, cu, lengths, table, q, some


@pytest.mark.parametrize("new,heads,dim,block", TILES)
@pytest.mark.parametrize("shifts", [(0, 4, 9), (0, 30, 60), (60, 30, 0), (5, 0, 40)],
                         ids=["rise", "rise far", "fall far", "both"])
def test_value_scales(new, heads, dim, block, shifts):
    announce(f"kv attention over segments, value scales {shifts}, {new} x {heads} rows of {dim}")
    ref, cu, lengths, table, q, some = segments(new, heads, dim, block, shifts)
    _kv_rows.compare(ref, ref.device(fp4), q, cu, lengths, table, heads=some, fp4=fp4)


@pytest.mark.parametrize("new,heads,dim,block", TILES)
@pytest.mark.parametrize("how", [{"window": 700}, {"window": 2500}, {"causal": False}],
                         ids=["window 700", "window 2500", "not causal"])
def test_windows(new, heads, dim, block, how):
    """Windows shorter and longer than a segment, and rows that see all."""
    announce(f"kv attention over segments, {how}, {new} x {heads} rows of {dim}")
    ref, cu, lengths, table, q, some = segments(new, heads, dim, block, (3, 0, 7))
    _kv_rows.compare(ref, ref.device(fp4), q, cu, lengths, table, heads=some, fp4=fp4, **how)


@pytest.mark.parametrize("new,heads,dim,block", TILES)
@pytest.mark.parametrize("how", [{}, {"window": 2300}, {"causal": False}],
                         ids=["causal", "window", "not causal"])
def test_nan_and_missing_pages(new, heads, dim, block, how):
    """In the second segment a NaN value and a page the cache does not have, in
    the third a NaN value that only some rows see."""
    announce(f"kv attention over segments with NaN and a missing page, {how}, {new} x {heads} rows "
             f"of {dim}")
    ref, cu, lengths, table, q, some = segments(new, heads, dim, block, (3, 0, 7))
    for p, d, code in ((2500, 5, 127), (4200 + new // 2, 9, 255)):
        ref.codes[1][table[0][p // block], 0, p % block, d] = code
    table[0][3000 // block] = -1
    _kv_rows.compare(ref, ref.device(fp4), q, cu, lengths, table, heads=some, fp4=fp4, **how)
