"""GPU test of the cache operators in use: the example attention layer, its
prompt and its single tokens, against the definition in 64 bits on the values
that the cache holds."""
import os
import sys

import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _kv
from tests._gpu import announce

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


class _Values:
    """What the reference needs of a cache: one sequence's values."""

    def __init__(self, k, v):
        self.kv = k, v

    def sequence(self, half, table, length):
        return self.kv[half][table[0]:table[0] + length]


def test_layer():
    import attention_layer
    layer = attention_layer.AttentionLayer(2048, heads=16, kv_heads=2, head_dim=128, device="cuda")
    seqs = attention_layer.Sequences(pages=24, kv_heads=2, block=32, head_dim=128, device="cuda")
    g = torch.Generator().manual_seed(0)
    for new in ([70, 33], [1, 1], [1, 0], [3, 2]):
        announce(f"attention layer, {new} new tokens")
        batch = seqs.extend(new)
        x = torch.randn(sum(new), 2048, generator=g).bfloat16().cuda()
        o = layer.attend(x, seqs.cache, batch)
        y = layer(x, seqs.cache, batch)  # writes the same rows again
        assert y.shape == x.shape and bool(y.isfinite().all())
        q = layer.project(x)[0].double().cpu().numpy()
        starts = np.concatenate([[0], np.cumsum(seqs.lengths)]).tolist()
        whole = (torch.tensor(starts, dtype=torch.int32, device="cuda"), *batch[1:])
        k, v = fp4.kv_cache_read(seqs.cache, *whole, starts[-1], out_dtype=torch.float32)
        values = _Values(k.double().cpu().numpy(), v.double().cpu().numpy())
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        want, _, weight, reach = _kv.attention(values, q, cu, seqs.lengths, [[s] for s in starts],
                                               128 ** -0.5)
        bound, _ = _kv.tolerance(weight, reach, want, max(seqs.lengths), 128, True)
        assert (np.abs(o.double().cpu().numpy() - want) <= bound).all()


def test_program(capsys):
    import attention_layer
    announce("attention layer example as a program")
    attention_layer.main()
    out = capsys.readouterr().out.splitlines()
    assert len(out) == 4 and "lengths [303, 80]" in out[3]
