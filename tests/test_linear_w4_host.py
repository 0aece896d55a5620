"""What the four-bit weight's linear layers refuse, before any HIP call (no GPU
is needed, pointers are never dereferenced)."""
import os

import pytest

import mxfp4_block_amax_amd as fp4

OK, E_ARG, E_SHAPE, E_DTYPE, E_ALIGN = 0, 1, 2, 3, 4
P = 0x10000

pytestmark = pytest.mark.skipif(not os.path.exists(fp4.LIB_PATH), reason="libfp4.so not built")


def rows(fmt=fp4.MXFP4, x=P, xt=fp4.BF16, m=4, k=512, codes=P, scales=P, s_g=P, n=64, c=P,
         ct=fp4.BF16):
    return fp4.lib().fp4_linear_w4(fmt, x, xt, m, k, codes, scales, s_g, n, c, ct, None)


def packed(fmt=fp4.MXFP4, x=P, xt=fp4.BF16, m=4, k=512, codes=P, s_g=P, n=64, c=P, ct=fp4.BF16):
    return fp4.lib().fp4_linear_w4_packed(fmt, x, xt, m, k, codes, s_g, n, c, ct, None)


@pytest.mark.parametrize("call", [rows, packed])
def test_refused(call):
    for null in ("x", "codes", "c"):
        assert call(**{null: None}) == E_ARG
    assert call(fmt=fp4.NVFP4, s_g=None) == E_ARG
    for bad in (-1, 2, 7):
        assert call(fmt=bad) == E_DTYPE and call(xt=bad) == E_DTYPE and call(ct=bad) == E_DTYPE
    for name in ("m", "n", "k"):
        for bad in (0, -1, -512, 2 ** 31, 2 ** 62):
            assert call(**{name: bad}) == E_SHAPE
    assert call(m=2 ** 19 + 1) == E_SHAPE and call(k=2 ** 20 + 512) == E_SHAPE
    assert call(n=2 ** 29, k=2 ** 19) == E_SHAPE
    for bad in (16, 40, 500):
        assert call(k=bad) == E_SHAPE
    assert call(x=P + 8) == E_ALIGN and call(codes=P + 8) == E_ALIGN
    assert call(c=P + 1) == E_ALIGN and call(c=P + 2, ct=fp4.F32) == E_ALIGN
    assert call(fmt=fp4.NVFP4, s_g=P + 2) == E_ALIGN


def test_blocks():
    assert rows(scales=None) == E_ARG
    assert rows(fmt=fp4.NVFP4, k=24) == E_SHAPE
    assert packed(k=256) == E_SHAPE and packed(fmt=fp4.NVFP4, k=768) == E_SHAPE
