"""GPU tests of attention over pages whose scale byte is 255: every value there
is NaN, zero codes included, for the rows that see the page and for no other."""
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _kv, _kv_rows
from tests import test_gpu_kv_attention as plain
from tests._gpu import announce

pytestmark = pytest.mark.gpu

# new tokens, group, dim, dtype: few rows, many rows, and fp32 queries
ROWS = [(1, 4, 64, "bf16"), (1, 4, 256, "fp32"), (6, 2, 128, "bf16"), (40, 1, 64, "bf16"),
        (40, 2, 128, "fp32"), (40, 1, 192, "bf16"), (40, 1, 256, "bf16"), (40, 1, 256, "fp32"),
        (100, 3, 64, "bf16"), (100, 8, 128, "bf16"), (100, 8, 192, "bf16"), (100, 8, 256, "bf16"),
        (520, 128, 64, "bf16"), (520, 255, 128, "bf16")]


@pytest.mark.parametrize("new,group,dim,dtype", ROWS)
@pytest.mark.parametrize("half", [0, 1], ids=["keys", "values"])
@pytest.mark.parametrize("zeros", [False, True], ids=["codes", "zeros"])
def test_nan_pages(new, group, dim, dtype, half, zeros):
    """Of one head: a page that a window hides from the later rows, and one that
    only the last rows see; then one that all of them see."""
    block, before = 32, 90
    ref, cu, lengths, table = plain.filled([new, 2], [before, 70], 2, block, dim)
    q = plain.queries(cu[-1], 2 * group, dim, dtype, 3)
    some = sorted({0, group - 1, group, 2 * group - 1})
    for where, window in (((before - 20, before + new - 1), 25), ((10,), 0)):
        for p in where:
            page = table[0][p // block]
            ref.scales[half][page, 0] = 255
            if zeros:
                ref.codes[half][page, 0] = 0
        announce(f"kv attention, pages of scale byte 255, half {half}, window {window}, {new} x "
                 f"{group} rows of {dim}, {dtype}")
        dev = ref.device(fp4)
        for batch in (_kv.batch(fp4, cu, lengths, table), _kv_rows.wide_batch(fp4, cu, lengths, table)):
            got, lse = _kv_rows.compare(ref, dev, q, cu, lengths, table, heads=some, fp4=fp4,
                                        batch=batch, window=window)
        assert bool(got[new - 1, :group].isnan().all()) and not bool(got[:, group:].isnan().any())
        assert bool(lse[new - 1, :group].isnan().all()) == (half == 0)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("half", [0, 1], ids=["keys", "values"])
def test_nan_page_of_steps_seen_whole(dim, half):
    """A page inside a step that every row sees, not causal and of zero codes."""
    for new, group, dtype in ((1, 4, "bf16"), (2, 4, "fp32"), (64, 16, "bf16")):
        ref, cu, lengths, table = plain.filled([new], [2048 - new], 1, 64, dim)
        page = table[0][9]
        ref.scales[half][page] = 255
        ref.codes[half][page] = 0
        q = plain.queries(new, group, dim, dtype, 4)
        announce(f"kv attention, a page of scale byte 255 seen whole, half {half}, {new} x {group} "
                 f"rows of {dim}, {dtype}")
        got, _ = _kv_rows.compare(ref, ref.device(fp4), q, cu, lengths, table, heads=[0, group - 1],
                                  fp4=fp4, causal=False)
        assert bool(torch.isnan(got).all())
