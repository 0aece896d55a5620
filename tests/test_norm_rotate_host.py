"""What the norm and rotation refuse, before any HIP call (no GPU is needed,
pointers are never dereferenced)."""
import os

import pytest

import mxfp4_block_amax_amd as fp4

OK, E_ARG, E_SHAPE, E_DTYPE, E_ALIGN = 0, 1, 2, 3, 4
P = 0x10000

pytestmark = pytest.mark.skipif(not os.path.exists(fp4.LIB_PATH), reason="libfp4.so not built")


def rows(x=P, y=P, xt=512, xh=128, yt=512, yh=128, weight=P, heads=4):
    return fp4._pack_head_rows(x, y, xt, xh, yt, yh, weight, heads)


def call(q=None, k=None, xt=fp4.BF16, wt=fp4.BF16, dim=128, eps=1e-6, cu=P, lengths=P, seqs=2,
         tokens=4, freq=P, rotary=128, interleaved=0, status=None):
    return fp4.lib().fp4_norm_rotate(q or rows(), k or rows(), xt, wt, dim, eps, cu, lengths, seqs,
                                     tokens, freq, rotary, interleaved, status, None)


def test_refused():
    lib = fp4.lib()
    assert lib.fp4_norm_rotate(None, rows(), 1, 1, 128, 0.0, P, P, 2, 4, P, 128, 0, None,
                               None) == E_ARG
    assert lib.fp4_norm_rotate(rows(), None, 1, 1, 128, 0.0, P, P, 2, 4, P, 128, 0, None,
                               None) == E_ARG
    for name in ("cu", "lengths", "freq"):
        assert call(**{name: None}) == E_ARG
    assert call(interleaved=2) == E_ARG
    for bad in (-1e-6, float("inf"), float("nan")):
        assert call(eps=bad) == E_ARG
    for bad in (-1, 2):
        assert call(xt=bad) == E_DTYPE and call(wt=bad) == E_DTYPE
    for bad in (0, 32, 80, 320, -128):
        assert call(dim=bad, rotary=16) == E_SHAPE
    for bad in (0, 8, 24, 144, -16):
        assert call(rotary=bad) == E_SHAPE
    for bad in (0, -1, 2 ** 20 + 1):
        assert call(seqs=bad) == E_SHAPE
    for bad in (-1, 2 ** 23 + 1, 2 ** 40):
        assert call(tokens=bad) == E_SHAPE
    assert call(cu=P + 2) == E_ALIGN and call(lengths=P + 1) == E_ALIGN
    assert call(freq=P + 4) == E_ALIGN and call(status=P + 2) == E_ALIGN
    assert call(tokens=0) == OK  # nothing to do


@pytest.mark.parametrize("side", ["q", "k"])
def test_rows(side):
    def one(**how):
        return call(**{side: rows(**how)})
    assert one(x=0) == E_ARG and one(y=0) == E_ARG
    for bad in (0, -1, 65536):
        assert one(heads=bad) == E_SHAPE
    for name in ("xh", "yh"):
        assert one(**{name: 127}) == E_SHAPE and one(**{name: 132}) == E_ALIGN
        assert one(**{name: 2 ** 62}) == E_SHAPE
    for name in ("xt", "yt"):
        assert one(**{name: -512}) == E_SHAPE and one(**{name: 516}) == E_ALIGN
        assert one(**{name: 2 ** 62}) == E_SHAPE
    for name in ("x", "y", "weight"):
        assert one(**{name: P + 8}) == E_ALIGN
