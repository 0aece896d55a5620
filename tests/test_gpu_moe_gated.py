"""The experts' gated values between the two products: all 24 bits of them, the largest
that fp32 holds, and infinities."""
import numpy as np
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests import _w4
from tests._gpu import announce

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ONE = {_w4.MX: 127, _w4.NV: 0x38}  # the scale byte of 1


def weight(fmt, code):
    """Codes [experts, rows, K] with scales of 1, as the calls take them."""
    packed = (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8)
    scales = np.full((*code.shape[:-1], code.shape[-1] // _w4.BLOCK[fmt]), ONE[fmt], dtype=np.uint8)
    parts = [torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda()]
    return parts + [torch.ones(code.shape[0], device="cuda")] * (fmt == _w4.NV)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("fmt", [_w4.MX, _w4.NV])
@pytest.mark.parametrize("tokens,inner", [(1, 32), (3, 512), (5, 1056), (17, 544), (40, 96),
                                          (70, 1600), (64, 2048)])
def test_all_bits(fmt, tokens, inner, dtype):
    """The gate is 32, whose silu is 32 in fp32 (exp(-32) is below 2^-24), the up values
    are sums of different powers of two, so whole numbers of 24 bits, and each row of the
    down projection takes one of them: every step is exact."""
    announce(f"moe_experts, bits of the gated values, {fmt} {tokens} {inner} {dtype}")
    g = np.random.default_rng(inner + tokens)
    experts, hidden = 4, inner
    up = np.zeros((experts, 2 * inner, hidden), dtype=np.int64)
    up[:, :inner, 24] = 2  # the code of 1
    bits = g.integers(0, 2, (experts, inner, 24))
    bits[..., 0] = bits[..., 23] = 1
    up[:, inner:, :24] = 2 * bits
    down = np.zeros((experts, hidden, inner), dtype=np.int64)
    place = np.stack([g.permutation(inner) for _ in range(experts)])
    down[np.arange(experts)[:, None], np.arange(hidden), place] = 2
    x = np.zeros((tokens, hidden))
    x[:, :24] = 2.0 ** (np.arange(24) + np.arange(tokens)[:, None] % 30)
    x[:, 24] = 32
    ids = g.integers(0, experts, (tokens, 1))
    value = bits @ 2 ** np.arange(24)
    want = 32.0 * value[ids, place[ids[:, 0]]] * 2.0 ** (np.arange(tokens) % 30)[:, None]
    got = fp4.moe_experts(fmt, torch.from_numpy(x).to(DTYPES[dtype]).cuda(),
                          torch.from_numpy(ids).int().cuda(), torch.ones(tokens, 1, device="cuda"),
                          weight(fmt, up), weight(fmt, down), out_dtype=torch.float32)
    assert np.array_equal(got.cpu().double().numpy(), want)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("fmt", [_w4.MX, _w4.NV])
@pytest.mark.parametrize("tokens", [2, 20])
def test_large_and_infinite(fmt, tokens, dtype):
    """2^128 - 2^118 is finite in fp32, but nearer to infinity than to any other value of
    bf16; 2^200 is infinite."""
    announce(f"moe_experts, large gated values, {fmt} {tokens} {dtype}")
    experts, hidden, inner = 2, 64, 32
    up = np.zeros((experts, 2 * inner, hidden), dtype=np.int64)
    up[:, 0, 0] = up[:, inner, 1] = 2   # gate and up of value 0: 2^100, 2^28
    up[:, inner, 2] = 10                # - 2^18
    up[1, inner, 3] = 2                 # + 2^100, of expert 1
    down = np.full((experts, hidden, inner), 2, dtype=np.int64)
    down[:, 1, 0], down[:, 2, 0], down[:, 3, 0] = 10, 0, 1  # -1, 0, 0.5
    x = np.zeros((tokens, hidden))
    x[:, 0], x[:, 1], x[:, 2], x[:, 3] = 2.0 ** 100, 2.0 ** 28, 2.0 ** 18, 2.0 ** 100
    ids = np.arange(tokens)[:, None] % 2
    got = fp4.moe_experts(fmt, torch.from_numpy(x).to(DTYPES[dtype]).cuda(),
                          torch.from_numpy(ids).int().cuda(),
                          torch.full((tokens, 1), 2.0 ** -10, device="cuda"),
                          weight(fmt, up), weight(fmt, down), out_dtype=torch.float32)
    got = got.cpu().double().numpy()
    large = np.full(hidden, 2.0 ** 118 - 2.0 ** 108)
    large[1], large[2], large[3] = -large[0], 0, large[0] / 2
    infinite = np.full(hidden, np.inf)
    infinite[1], infinite[2] = -np.inf, np.nan
    assert np.array_equal(got[0::2], np.broadcast_to(large, got[0::2].shape))
    assert np.array_equal(got[1::2], np.broadcast_to(infinite, got[1::2].shape), equal_nan=True)
