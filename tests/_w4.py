"""FP4 weights and what is multiplied with them, in 64 bits on the CPU, from the
formats' definition.  Test infrastructure; shares nothing with the library."""
import math

import numpy as np
import torch

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
E8M0 = np.array([2.0 ** (b - 127) for b in range(255)] + [math.nan])
E4M3 = np.array([math.ldexp(b & 7, -9) if b < 8 else math.ldexp(8 + (b & 7), (b >> 3) - 10)
                 for b in range(127)] + [math.nan])
E4M3 = np.concatenate([E4M3, -E4M3])
MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}


class Weight:
    """[.., rows, K] codes and scales; s_g a float32 vector over the leading index."""

    def __init__(self, fmt, codes, scales, s_g=None):
        self.fmt, self.codes, self.scales, self.s_g = fmt, codes, scales, s_g

    def values(self, at=None):
        """[rows, K] float64 without the tensor scale (of leading index `at`)."""
        codes = self.codes if at is None else self.codes[at]
        scales = self.scales if at is None else self.scales[at]
        v = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]))
        v[..., 0::2], v[..., 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
        s = (E8M0 if self.fmt == MX else E4M3)[scales]
        return v * np.repeat(s, BLOCK[self.fmt], -1)

    def factor(self, at=0):
        return 1.0 if self.s_g is None else float(self.s_g[at])

    def device(self):
        put = lambda a: torch.from_numpy(a.copy()).cuda()
        return put(self.codes), put(self.scales), None if self.s_g is None else put(self.s_g)


def exact_weight(fmt, shape, g):
    """Random codes, and scales within a few powers of two: its products with
    small integers are multiples of 2^-6 below 2^9, so that sums of some
    thousands of them are exact in fp32 whatever their order."""
    codes = g.integers(0, 256, (*shape[:-1], shape[-1] // 2)).astype(np.uint8)
    at = (*shape[:-1], shape[-1] // BLOCK[fmt])
    if fmt == MX:
        return Weight(fmt, codes, g.integers(124, 129, at).astype(np.uint8))
    # +-(8 .. 15) 2^-4 .. 2^-3 and zero
    scales = g.integers(0x30, 0x40, at) + 128 * g.integers(0, 2, at)
    scales[g.random(at) < 0.05] = 0
    return Weight(fmt, codes, scales.astype(np.uint8),
                  np.full(math.prod(shape[:-2]), 0.25, dtype=np.float32))


def wide_weight(fmt, shape, g):
    """Random codes, scales over a wide range, any tensor scale."""
    codes = g.integers(0, 256, (*shape[:-1], shape[-1] // 2)).astype(np.uint8)
    at = (*shape[:-1], shape[-1] // BLOCK[fmt])
    if fmt == MX:
        return Weight(fmt, codes, g.integers(100, 125, at).astype(np.uint8))
    return Weight(fmt, codes, (g.integers(0, 127, at) + 128 * g.integers(0, 2, at)).astype(np.uint8),
                  g.uniform(1e-5, 1e-3, math.prod(shape[:-2])).astype(np.float32))


def product_bound(roundings, size):
    """What a sum of exact products may be off by: `roundings` fp32 additions lie
    between a product and the sum, each off by at most 2^-23 (a matrix
    instruction may cut rather than round) of what is added up, below `size`, the
    sum of magnitudes."""
    return roundings * 2.0 ** -23 * size


def output_eps(dtype):
    return torch.finfo(dtype).eps / 2
