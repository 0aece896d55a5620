"""Norms of heads whose squares fp32 does not hold."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests._gpu import announce
from tests.test_gpu_norm_rotate import DTYPES, batch_of, check, frequencies, reference

pytestmark = pytest.mark.gpu


def check_where_defined(got, want, size, dtype):
    """Zeros over zero (a head of zeros, without eps) are NaN, and nothing else is."""
    got, undefined = got.cpu().clone(), want.isnan()
    assert torch.equal(got.isnan(), undefined)
    got[undefined] = 0
    check(got, want.nan_to_num(0.0), size.nan_to_num(0.0), dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-35, 1e-12, 1e-6, 1e30, 3e38])
def test_large_and_small(dim, eps, interleaved, dtype):
    """Heads of all sizes side by side in a wave, up to the largest values and down to
    those below the normal range; one value far above the others; zeros."""
    announce(f"norm_rotate far values {dim} {eps} {interleaved} {dtype}")
    g = torch.Generator().manual_seed(dim)
    sizes = [1e25, 1.0, 1e-25, 3e38, 1e-38, 1e19, 1e-19, 1e-12, 2e-40, 1e10, 6e18]
    x = torch.rand(9, 2 * len(sizes), dim, generator=g, dtype=torch.float64) * 2 - 1
    x *= torch.tensor(sizes + sizes[::-1], dtype=torch.float64)[:, None]
    x[3, :, 5] *= 1e-30
    x[4, :, :dim - 1] *= 1e-9
    if eps:
        x[5, 3::5] = 0
    x = x.to(DTYPES[dtype])
    assert x.isfinite().all()
    w = (1 + 0.3 * torch.randn(2, dim, generator=g)).to(DTYPES[dtype])
    cu, lengths, pos = batch_of([4, 5], [3, 70])
    freq = frequencies(dim)
    kv = x[:, 5:9].contiguous()
    q, k = fp4.norm_rotate(x.cuda(), kv.cuda(), cu.cuda(), lengths.cuda(), freq.cuda(), w[0].cuda(),
                           w[1].cuda(), eps=eps, interleaved=interleaved)
    eps = float(np.float32(eps))
    check_where_defined(q, *reference(x, w[0], pos, freq, eps, interleaved), DTYPES[dtype])
    check_where_defined(k, *reference(kv, w[1], pos, freq, eps, interleaved), DTYPES[dtype])
    # and of queries alone: keys as they are
    q2, k2 = fp4.norm_rotate(x.cuda(), kv.cuda(), cu.cuda(), lengths.cuda(), freq.cuda(),
                             w[0].cuda(), eps=eps, interleaved=interleaved)
    _, plain = fp4.norm_rotate(x.cuda(), kv.cuda(), cu.cuda(), lengths.cuda(), freq.cuda(),
                               interleaved=interleaved)
    assert torch.equal(q2.nan_to_num(7.0), q.nan_to_num(7.0)) and torch.equal(k2, plain)
