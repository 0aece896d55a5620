"""GPU tests of attention over the 8-bit cache against bounds for weights of 11
bits (bf16 queries) and 22 bits (fp32): the cases of the other files, whose
bounds for bf16 queries are wider."""
import pytest

import mxfp4_block_amax_amd as fp4
from tests import _kv_rows
from tests import test_gpu_kv_attention as plain
from tests import test_gpu_kv_attention_tiles as tiles
from tests._gpu import announce

pytestmark = pytest.mark.gpu


def both_tables(ref, q, cu, lengths, table, **how):
    dev = ref.device(fp4)
    for batch in (None, _kv_rows.wide_batch(fp4, cu, lengths, table)):
        _kv_rows.compare(ref, dev, q, cu, lengths, table, fp4=fp4, batch=batch, **how)


@pytest.mark.parametrize("heads,group,block,dim,dtype,new,before", plain.CASES + tiles.CASES)
def test_causal(heads, group, block, dim, dtype, new, before):
    announce(f"kv attention, close bounds, {heads}x{group} heads, pages of {block} x {dim}, {dtype}, "
             f"{new} after {before}")
    ref, cu, lengths, table = plain.filled(new, before, heads, block, dim)
    q = plain.queries(cu[-1], heads * group, dim, dtype, 1)
    both_tables(ref, q, cu, lengths, table)
    both_tables(ref, q, cu, lengths, table, causal=False)
    both_tables(ref, q, cu, lengths, table, window=50)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("seqs,top", [(1, 2), (65, 8), (255, 8), (256, 8), (300, 8), (65, 90)])
def test_many_sequences(seqs, top, dtype):
    new, before = tiles.many(seqs, top)
    if seqs == 1:
        new, before = [1], [1000]
    ref, cu, lengths, table = plain.filled(new, before, 1, 16, 64)
    q = plain.queries(cu[-1], 3, 64, dtype, 3)
    announce(f"kv attention, close bounds, {seqs} sequences of up to {top} tokens, {dtype}")
    _kv_rows.compare(ref, ref.device(fp4), q, cu, lengths, table, fp4=fp4)
