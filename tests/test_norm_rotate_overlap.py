"""Outputs whose tokens lie over each other are refused; inputs may (no GPU is needed,
pointers are never dereferenced)."""
import os

import pytest

import mxfp4_block_amax_amd as fp4
from tests.test_norm_rotate_host import E_SHAPE, call, rows

pytestmark = pytest.mark.skipif(not os.path.exists(fp4.LIB_PATH), reason="libfp4.so not built")


@pytest.mark.parametrize("side", ["q", "k"])
def test_refused(side):
    for stride in (0, 8, 120):
        assert call(**{side: rows(yt=stride)}) == E_SHAPE
        assert call(**{side: rows(yt=stride)}, tokens=2) == E_SHAPE
    # the check behind it is reached with strides that are good
    for good in (128, 512):
        assert call(**{side: rows(yt=good, weight=0x10008)}) not in (E_SHAPE, 0)
    assert call(**{side: rows(xt=0, weight=0x10008)}) not in (E_SHAPE, 0)
    assert call(**{side: rows(yt=0, weight=0x10008)}, tokens=1) not in (E_SHAPE, 0)
