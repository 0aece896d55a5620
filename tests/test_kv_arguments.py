"""CPU tests of what the Python cache calls hand to the library: a recording
stand-in for the library, host tensors in the place of device ones."""
import ctypes

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

    fp4_kv_cache_write = fp4_kv_cache_read = fp4_kv_attention = _call

    def fp4_kv_attention_workspace_bytes(self, *args):
        self.calls.append(args)
        return 64


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(fp4, "_lib", lib)
    monkeypatch.setattr(fp4, "_raw_stream", lambda device: 0)
    return lib


def host_cache(monkeypatch):
    """A cache of host tensors: the constructor takes device ones."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    u8 = torch.uint8
    return fp4.KVCache(torch.zeros(4, 2, 16, 64, dtype=u8), torch.zeros(4, 2, dtype=u8),
                       torch.zeros(4, 2, 16, 64, dtype=u8), torch.zeros(4, 2, dtype=u8))


@pytest.fixture
def cache(library, monkeypatch):
    return host_cache(monkeypatch)


BATCH = [torch.tensor(a, dtype=torch.int32) for a in ([0, 3], [3], [[1]])]
K = torch.zeros(3, 2, 64)
Q = torch.zeros(3, 4, 64)


def write(cache, **how):
    fp4.kv_cache_write(cache, K, K, *BATCH, **how)


def read(cache, **how):
    fp4.kv_cache_read(cache, *BATCH, 3, **how)


def attend(cache, **how):
    fp4.kv_attention(Q, cache, *BATCH, **how)


@pytest.mark.parametrize("call", [write, read, attend])
@pytest.mark.parametrize("check", [False, True])
def test_status_of_another_kind(call, check, cache, library):
    """The kernels write 4 bytes through its pointer."""
    for bad in (torch.zeros(1, dtype=torch.int32, device="meta"),  # another device's
                torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int64),
                torch.zeros(1)):
        with pytest.raises((TypeError, ValueError)):
            call(cache, check=check, status=bad)
    assert not [c for c in library.calls if len(c) > 5]  # none reached a launch
    call(cache, check=check, status=torch.zeros(1, dtype=torch.int32))
    call(cache, check=False)
    assert len([c for c in library.calls if len(c) > 5]) == 2


def test_workspace_of_another_kind(cache, library):
    """The kernels write its bytes in one piece."""
    for bad in (torch.zeros(64, dtype=torch.uint8, device="meta"),
                torch.zeros(64, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError):
            attend(cache, check=False, workspace=bad)
    assert not library.calls


def test_workspace_size_in_bytes(cache, library):
    for space in (torch.zeros(64, dtype=torch.uint8), torch.zeros(4, 4)):
        attend(cache, check=False, workspace=space)
        pointer, size = library.calls[-1][12:14]
        assert (pointer, size) == (space.data_ptr(), 64)


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 80])
def test_windows_past_32_bits(window, cache, library):
    """The library takes 32 bits: a window longer than any sequence stays one."""
    attend(cache, check=False, window=window)
    for at, call in ((9, library.calls[-1]), (3, library.calls[-2])):  # attention; its workspace
        assert ctypes.c_int32(call[at]).value >= 2 ** 27
    attend(cache, check=False, window=-window)
    assert ctypes.c_int32(library.calls[-1][9]).value < 0  # for the library to refuse


def test_a_cache_keeps_its_tensors(cache):
    """The calls use their addresses: another tensor makes another cache."""
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        held = getattr(cache, name)
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.zeros_like(held))
        assert getattr(cache, name) is held
