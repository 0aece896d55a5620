"""Small fp32 activations: all bits down to 2^-110, below that those from 2^-133 on."""
import numpy as np
import pytest
import torch

from tests import _w4
from tests._gpu import announce
from tests.test_gpu_linear_w4 import layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["rows", "packed"])
@pytest.mark.parametrize("m", [4, 8, 16, 33])
def test_bits(m, layout):
    announce(f"linear_w4 small activations {m} {layout}")
    g = np.random.default_rng(m)
    k, n = 1024, 40
    codes = g.integers(1, 8, (n, k // 2)) * 17  # both values of a byte alike, no zeros
    w = _w4.Weight(_w4.MX, codes.astype(np.uint8), np.full((n, k // 32), 127 + 100, dtype=np.uint8))
    exponent = np.concatenate([[-133, -134, -135, -140, -156, -126 - 23, -128, -133],
                               g.integers(-165, -120, m)])[:m]
    # one activation a row: 24 random bits times 2^exponent, as fp32 holds it
    value = (g.integers(2 ** 23, 2 ** 24, m) * 2.0 ** exponent).astype(np.float32)
    value *= g.choice([-1, 1], m).astype(np.float32)
    at = (np.arange(m) * 131 + 7) % k
    x = torch.zeros(m, k)
    x[torch.arange(m), torch.from_numpy(at)] = torch.from_numpy(value)
    held = np.trunc(value.astype(np.float64) * 2.0 ** 133) * 2.0 ** -133
    assert (held == value)[np.abs(value) >= 2.0 ** -110].all() and (held != value).any()
    want = held[:, None] * w.values()[:, at].T
    got = layer(layout, w, x.cuda()).cpu().double().numpy()
    # three products at one place: two roundings
    assert (np.abs(got - want) <= 2 * 2.0 ** -23 * np.abs(want)).all()
