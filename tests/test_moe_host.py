"""What the calls of a mixture of experts refuse, before any HIP call (no GPU is
needed, pointers are never dereferenced)."""
import os

import pytest

import mxfp4_block_amax_amd as fp4

OK, E_ARG, E_SHAPE, E_DTYPE, E_ALIGN, E_WORKSPACE = 0, 1, 2, 3, 4, 5
P = 0x10000

pytestmark = pytest.mark.skipif(not os.path.exists(fp4.LIB_PATH), reason="libfp4.so not built")


def route(x=P, xt=fp4.BF16, tokens=4, hidden=64, router=P, rt=fp4.F32, experts=16, top_k=2,
          renormalize=1, chosen=P, weights=P, ws=P, wsb=2 ** 40):
    return fp4.lib().fp4_moe_route(x, xt, tokens, hidden, router, rt, experts, top_k, renormalize,
                                   chosen, weights, ws, wsb, None)


def test_route():
    for null in ("x", "router", "chosen", "weights"):
        assert route(**{null: None}) == E_ARG
    assert route(renormalize=2) == E_ARG
    assert route(xt=2) == E_DTYPE and route(rt=-1) == E_DTYPE
    for bad in (0, -1, 2 ** 20 + 1, 2 ** 62):
        assert route(tokens=bad) == E_SHAPE
    for bad in (0, -8, 4, 12, 2 ** 40):
        assert route(hidden=bad) == E_SHAPE
    for bad in (0, -1, 1025):
        assert route(experts=bad) == E_SHAPE
    assert route(top_k=0) == E_SHAPE and route(top_k=17) == E_SHAPE
    assert route(experts=64, top_k=33) == E_SHAPE
    for name in ("x", "router", "ws"):
        assert route(**{name: P + 8}) == E_ALIGN
    assert route(chosen=P + 2) == E_ALIGN and route(weights=P + 1) == E_ALIGN
    space = fp4.lib().fp4_moe_route_workspace_bytes
    need = space(4, 64, 16)
    assert need >= 4 * 16 * 8
    assert route(wsb=need - 1) == E_WORKSPACE and route(ws=None) == E_WORKSPACE
    for bad in ((0, 64, 16), (4, 63, 16), (4, 64, 0), (4, 64, 1025), (2 ** 40, 64, 16),
                (4, -64, 16)):
        assert space(*bad) == 0


def weights(uc=P, us=P, dc=P, ds=P, ug=P, dg=P, hidden=64, inner=96, experts=8, stride=0):
    return fp4._pack_moe_weights(uc, us, dc, ds, ug, dg, hidden, inner, experts, stride)


def experts(fmt=fp4.MXFP4, w=None, x=P, xt=fp4.BF16, tokens=4, ids=P, share=P, top_k=2, out=P,
            ot=fp4.BF16, ws=P, wsb=2 ** 40, status=None):
    return fp4.lib().fp4_moe_experts(fmt, w or weights(), x, xt, tokens, ids, share, top_k, out, ot,
                                     ws, wsb, status, None)


@pytest.mark.parametrize("fmt", [fp4.MXFP4, fp4.NVFP4])
def test_experts(fmt):
    def call(**how):
        return experts(fmt=fmt, **how)
    lib = fp4.lib()
    assert lib.fp4_moe_experts(fmt, None, P, 1, 4, P, P, 2, P, 1, P, 2 ** 40, None, None) == E_ARG
    for null in ("uc", "us", "dc", "ds"):
        assert call(w=weights(**{null: 0})) == E_ARG
    for null in ("x", "ids", "share", "out"):
        assert call(**{null: None}) == E_ARG
    for bad in (-1, 2):
        assert experts(fmt=bad) == E_DTYPE and call(xt=bad) == E_DTYPE and call(ot=bad) == E_DTYPE
        assert call(w=weights(stride=bad)) == E_ARG
    for bad in (0, -1, 2 ** 20 + 1, 2 ** 62):
        assert call(tokens=bad) == E_SHAPE
    for bad in (0, -1, 33):
        assert call(top_k=bad) == E_SHAPE
    for bad in (0, -32, 8, 40, 2 ** 40):
        assert call(w=weights(hidden=bad)) == E_SHAPE and call(w=weights(inner=bad)) == E_SHAPE
    for bad in (0, -1, 1025):
        assert call(w=weights(experts=bad)) == E_SHAPE
    assert call(w=weights(hidden=2 ** 20, inner=2 ** 11)) == E_SHAPE
    assert call(w=weights(inner=2 ** 16 + 32)) == E_SHAPE
    for name in ("uc", "dc"):
        assert call(w=weights(**{name: P + 8})) == E_ALIGN
    assert call(x=P + 8) == E_ALIGN and call(ws=P + 8) == E_ALIGN and call(ids=P + 2) == E_ALIGN
    assert call(share=P + 2) == E_ALIGN and call(out=P + 1) == E_ALIGN
    assert call(out=P + 2, ot=fp4.F32) == E_ALIGN and call(status=P + 2) == E_ALIGN
    space = lib.fp4_moe_experts_workspace_bytes
    need = space(weights(), fmt, 4, 2, fp4.BF16)
    assert need == 4 * 2 * 96 * 4
    assert call(wsb=need - 1) == E_WORKSPACE and call(ws=None) == E_WORKSPACE
    for bad in ((None, fmt, 4, 2, 1), (weights(), 2, 4, 2, 1), (weights(), fmt, 0, 2, 1),
                (weights(), fmt, 4, 0, 1), (weights(), fmt, 4, 2, 2),
                (weights(inner=24), fmt, 4, 2, 1)):
        assert space(*bad) == 0


def test_blocks_and_tensor_scales():
    assert experts(w=weights(hidden=48)) == E_SHAPE  # whole blocks of NVFP4 alone
    assert experts(fmt=fp4.NVFP4, w=weights(ug=0)) == E_ARG
    assert experts(fmt=fp4.NVFP4, w=weights(dg=0)) == E_ARG
    assert experts(fmt=fp4.NVFP4, w=weights(ug=P + 2)) == E_ALIGN
