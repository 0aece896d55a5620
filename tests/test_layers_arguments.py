"""CPU tests of what the decoding layers' Python calls refuse and hand to the
library: a recording stand-in for the library, host tensors in the place of device
ones."""
import pytest
import torch

import mxfp4_block_amax_amd as fp4


class Library:
    """Records the entry points' arguments."""

    def __init__(self):
        self.calls = []

    def _call(self, *args):
        self.calls.append(args)
        return 0

    fp4_linear_w4 = fp4_linear_w4_packed = fp4_moe_route = fp4_moe_experts = fp4_norm_rotate = _call

    def _size(self, *args):
        return 64

    fp4_moe_route_workspace_bytes = fp4_moe_experts_workspace_bytes = _size

    def fp4_packed_operand_bytes(self, rows, k):
        return rows * k // 2 if k % 512 == 0 else 0

    fp4_nv_packed_operand_bytes = fp4_packed_operand_bytes


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(fp4, "_lib", lib)
    monkeypatch.setattr(fp4, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(fp4, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0 if t.device.type == "cpu" else 1)
    return lib


U8 = torch.uint8
X = torch.zeros(2, 3, 64)
CODES, SCALES = torch.zeros(5, 32, dtype=U8), torch.zeros(5, 2, dtype=U8)
NV_SCALES, S_G = torch.zeros(5, 4, dtype=U8), torch.ones(1)


def test_linear(library):
    y = fp4.linear_w4(fp4.MXFP4, X, CODES, SCALES)
    assert y.shape == (2, 3, 5) and y.dtype == torch.float32
    assert library.calls[-1][:8] == (0, X.data_ptr(), fp4.F32, 6, 64, CODES.data_ptr(),
                                     SCALES.data_ptr(), None)
    assert library.calls[-1][8:] == (5, y.data_ptr(), fp4.F32, 0)
    y = fp4.linear_w4(fp4.NVFP4, X.bfloat16(), CODES, NV_SCALES, S_G, out_dtype=torch.float32)
    assert library.calls[-1][2] == fp4.BF16 and library.calls[-1][7] == S_G.data_ptr()
    assert y.dtype == torch.float32
    n = len(library.calls)
    assert fp4.linear_w4(fp4.MXFP4, X[:, :0], CODES, SCALES).shape == (2, 0, 5)
    meta = torch.zeros(5, 32, dtype=U8, device="meta")
    for bad, error in (
            ((2, X, CODES, SCALES), ValueError), ((0, X[..., :32], CODES, SCALES), ValueError),
            ((0, X.transpose(0, 1), CODES, SCALES), ValueError),
            ((0, X.half(), CODES, SCALES), TypeError), ((0, X.double(), CODES, SCALES), TypeError),
            ((0, X, CODES.float(), SCALES), TypeError), ((0, X, CODES[0], SCALES), ValueError),
            ((0, X, CODES, NV_SCALES), ValueError), ((0, X, meta, SCALES), ValueError),
            ((1, X, CODES, NV_SCALES), TypeError), ((1, X, CODES, NV_SCALES, 1.0), TypeError),
            ((1, X, CODES, NV_SCALES, S_G[:0]), ValueError),
            ((1, X, CODES, NV_SCALES, S_G.double()), TypeError)):
        with pytest.raises(error):
            fp4.linear_w4(*bad)
    for out in (torch.zeros(2, 3, 6), torch.zeros(2, 5, 3).transpose(1, 2),
                torch.zeros(2, 3, 5, device="meta")):
        with pytest.raises(ValueError):
            fp4.linear_w4(0, X, CODES, SCALES, out=out)
    with pytest.raises(ValueError):
        fp4.linear_w4(0, X, CODES, SCALES, out=torch.zeros(2, 3, 5), out_dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fp4.linear_w4(0, X, CODES, SCALES, out=torch.zeros(2, 3, 5).half())
    assert len(library.calls) == n


def test_linear_packed(library):
    x, packed = torch.zeros(3, 512), torch.zeros(5 * 256, dtype=U8)
    y = fp4.linear_w4_packed(0, x, packed, 5)
    assert y.shape == (3, 5) and library.calls[-1][3:7] == (3, 512, packed.data_ptr(), None)
    n = len(library.calls)
    for bad in ((0, x, packed, 6), (0, torch.zeros(3, 256), packed, 5), (3, x, packed, 5),
                (0, x, torch.zeros(10 * 256, dtype=U8)[::2], 5)):
        with pytest.raises(ValueError):
            fp4.linear_w4_packed(*bad)
    for bad in ((1, x, packed, 5), (0, x, packed.view(torch.int8), 5)):
        with pytest.raises(TypeError):
            fp4.linear_w4_packed(*bad)
    assert len(library.calls) == n


def test_route(library):
    x, router = torch.zeros(4, 16).bfloat16(), torch.zeros(8, 16)
    ids, weights = fp4.moe_route(x, router, 2, renormalize=False)
    assert ids.dtype == torch.int32 and weights.dtype == torch.float32
    assert ids.shape == weights.shape == (4, 2)
    call = library.calls[-1]
    assert call[1:9] == (fp4.BF16, 4, 16, router.data_ptr(), fp4.F32, 8, 2, 0)
    n = len(library.calls)
    assert fp4.moe_route(x[:0], router, 2)[0].shape == (0, 2)
    for bad in ((x[:, :8], router, 2), (x, router[0], 2), (x, router, 0), (x, router, 9),
                (x, router.t().contiguous().t(), 2), (x, torch.zeros(8, 16, device="meta"), 2)):
        with pytest.raises(ValueError):
            fp4.moe_route(*bad)
    for out in ((ids.long(), weights), (ids, weights.double()), (ids[:3], weights),
                (ids, torch.zeros(2, 4).t())):
        with pytest.raises(ValueError):
            fp4.moe_route(x, router, 2, out=out)
    with pytest.raises(ValueError):
        fp4.moe_route(x, router, 2, workspace=torch.zeros(64, dtype=U8, device="meta"))
    assert len(library.calls) == n


def expert_weights(fmt=0, experts=3, hidden=64, inner=32, scales=None):
    block = 16 if fmt else 32
    make = lambda r, k: (torch.zeros(experts, r, k // 2, dtype=U8),
                         torch.zeros(experts, r, k // block, dtype=U8))
    up, down = make(2 * inner, hidden), make(hidden, inner)
    return (up, down) if scales is None else ((*up, torch.ones(scales)), (*down, torch.ones(scales)))


def test_experts(library):
    x, ids, w = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    y = fp4.moe_experts(0, x, ids, w, *expert_weights())
    assert y.shape == (4, 64) and len(library.calls[-1][1]) == 72
    assert library.calls[-1][3:5] == (fp4.F32, 4) and library.calls[-1][7] == 2
    for scales in (1, 3):
        fp4.moe_experts(1, x, ids, w, *expert_weights(1, scales=scales), check=False)
        assert library.calls[-1][12] is None
    n = len(library.calls)
    assert fp4.moe_experts(0, x[:0], ids[:0], w[:0], *expert_weights()).shape == (0, 64)
    up, down = expert_weights()
    for bad in ((2, x, ids, w, up, down), (0, x, ids[:3], w, up, down), (0, x, ids, w[:, :1], up, down),
                (0, x, ids.t().contiguous().t(), w, up, down), (0, x[:, :32], ids, w, up, down),
                (0, x, ids, w, up, expert_weights(experts=2)[1]),
                (0, x, ids, w, expert_weights(inner=64)[0], down),
                (0, x, ids, w, (up[0], up[1][:, :, :1]), down),
                (1, x, ids, w, *expert_weights(1)), (1, x, ids, w, *expert_weights(1, scales=2))):
        with pytest.raises(ValueError):
            fp4.moe_experts(*bad)
    for bad in ((0, x, ids.long(), w, up, down), (0, x, ids, w.double(), up, down),
                (0, x.half(), ids, w, up, down)):
        with pytest.raises(TypeError):
            fp4.moe_experts(*bad)
    for how in (dict(status=torch.zeros(0, dtype=torch.int32)), dict(out=torch.zeros(4, 32)),
                dict(workspace=torch.zeros(64, 2, dtype=U8)[:, 0])):
        with pytest.raises(ValueError):
            fp4.moe_experts(0, x, ids, w, up, down, **how)
    assert len(library.calls) == n


def test_rotate(library):
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)
    qkv = torch.zeros(3, 6, 64)
    q, k, freq = qkv[:, :4], qkv[:, 4:5], torch.zeros(32, dtype=torch.float64)
    out = fp4.norm_rotate(q, k, i32(0, 3), i32(7), freq, torch.ones(64), torch.ones(64))
    assert [t.shape for t in out] == [q.shape, k.shape] and all(t.is_contiguous() for t in out)
    assert fp4.norm_rotate(q, k, i32(0, 3), i32(7), freq, out=(q, k)) == (q, k)
    n = len(library.calls)
    for bad in ((q, k[:2], i32(0, 3), i32(7), freq), (q, k[..., :32], i32(0, 3), i32(7), freq),
                (q, k.bfloat16(), i32(0, 3), i32(7), freq), (q, k, i32(0, 3), i32(7, 8), freq),
                (q, k, i32(0, 1, 2, 3)[::2], i32(7), freq), (q, k, i32(0, 3), i32(7), freq[None]),
                (q[0], k, i32(0, 3), i32(7), freq),
                (q, k, i32(0, 3), i32(7), freq, torch.ones(32)),
                (q, k, i32(0, 3), i32(7), freq, torch.ones(64), torch.ones(64).bfloat16()),
                (q.transpose(1, 2).contiguous().transpose(1, 2), k, i32(0, 3), i32(7), freq)):
        with pytest.raises(ValueError):
            fp4.norm_rotate(*bad)
    for bad in ((q, k, i32(0, 3).long(), i32(7), freq), (q, k, i32(0, 3), i32(7), freq.float()),
                (q.half(), k.half(), i32(0, 3), i32(7), freq)):
        with pytest.raises(TypeError):
            fp4.norm_rotate(*bad)
    for out in ((q[:2], k), (q, k.bfloat16()), (q.to("meta"), k)):
        with pytest.raises((ValueError, TypeError)):
            fp4.norm_rotate(q, k, i32(0, 3), i32(7), freq, out=out)
    assert len(library.calls) == n
