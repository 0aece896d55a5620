"""GPU tests of the cache calls on batches of tens of thousands of sequences:
more work items than a grid's second dimension takes, and searches of three
steps."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _kv
from tests._gpu import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,most", [(40000, 1), (70000, 1), (70000, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_have_their_own_values(seqs, most, dtype):
    """Written, read back, and attended to with a window of one token: every row
    gets what was written for it, exactly but for attention of fp32 queries, whose
    one weight is rounded to 22 bits and divided by itself unrounded."""
    g = np.random.default_rng(seqs + most)
    new = g.integers(0, most + 1, seqs) if most > 1 else np.ones(seqs, dtype=np.int64)
    cu = np.concatenate([[0], np.cumsum(new)])
    batch = _kv.batch(fp4, cu, new, g.permutation(seqs)[:, None])
    rows = int(cu[-1])
    announce(f"kv write, read and attention of {seqs} sequences of up to {most} tokens, {dtype}")
    dev = fp4.new_kv_cache(seqs, 1, 16, 64, "cuda")
    # integers to 15 are E4M3 values under every scale that a page of them has
    t = torch.arange(rows, device="cuda")
    x = ((t[:, None] >> (3 * (torch.arange(64, device="cuda") % 7))) & 7).to(dtype)[:, None]
    fp4.kv_cache_write(dev, x, x + 8, *batch)
    k, v = fp4.kv_cache_read(dev, *batch, rows, out_dtype=dtype)
    assert torch.equal(k, x) and torch.equal(v, x + 8)
    q = torch.randn(rows, 2, 64, device="cuda").to(dtype)
    out, lse = fp4.kv_attention(q, dev, *batch, window=1, return_lse=True)
    if dtype is torch.bfloat16:
        assert torch.equal(out, (x + 8).expand(-1, 2, -1))
    else:
        assert bool(((out - x - 8).abs() <= (x + 8) * (2.0 ** -22 + 34 * 2.0 ** -24)).all())
    want = (q.double() * x.double()).sum(-1) * 64 ** -0.5
    assert bool(((lse - want).abs() <= 2.0 ** -24 * (136 * 64 * 7 + 16) * q.abs().amax(-1)).all())
