"""Host-side tests of the cache entry points: arguments they must refuse, before
any HIP call (no GPU is needed, pointers are never dereferenced), and the same
under AddressSanitizer and UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

import mxfp4_block_amax_amd as fp4
from mxfp4_block_amax_amd import build as fp4_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, E_ARG, E_SHAPE, E_DTYPE, E_ALIGN, E_WORKSPACE = 0, 1, 2, 3, 4, 5
P = 0x10000

pytestmark = pytest.mark.skipif(not os.path.exists(fp4.LIB_PATH), reason="libfp4.so not built")


def cache(kc=P, ks=P, vc=P, vs=P, pages=8, heads=2, block=16, dim=64):
    return fp4._pack_kv_cache(kc, ks, vc, vs, pages, heads, block, dim)


def batch(cu=P, lengths=P, table=P, tokens=4, stride=3, seqs=2, width=3):
    return fp4._pack_kv_batch(cu, lengths, table, tokens, stride, seqs, width)


def write(c=None, b=None, k=P, kt=128, kh=64, v=P, vt=128, vh=64, dt=fp4.BF16, status=None):
    return fp4.lib().fp4_kv_cache_write(c or cache(), b or batch(), k, kt, kh, v, vt, vh, dt,
                                        status, None)


def read(c=None, b=None, k=P, v=P, dt=fp4.BF16, status=None):
    return fp4.lib().fp4_kv_cache_read(c or cache(), b or batch(), k, v, dt, status, None)


def attend(c=None, b=None, q=P, qt=256, qh=64, dt=fp4.BF16, heads=4, scale=0.125, causal=1,
           window=0, out=P, lse=None, ws=None, wsb=0, status=None):
    return fp4.lib().fp4_kv_attention(c or cache(), b or batch(), q, qt, qh, dt, heads, scale,
                                      causal, window, out, lse, ws, wsb, status, None)


def space(c=None, b=None, heads=4, window=0, dt=fp4.BF16):
    return fp4.lib().fp4_kv_attention_workspace_bytes(c or cache(), b or batch(), heads, window, dt)


@pytest.mark.parametrize("call", [write, read, attend])
def test_cache_and_batch(call):
    lib = fp4.lib()
    assert lib.fp4_kv_cache_read(None, batch(), P, P, fp4.BF16, None, None) == E_ARG
    assert lib.fp4_kv_cache_read(cache(), None, P, P, fp4.BF16, None, None) == E_ARG
    for null in ("kc", "ks", "vc", "vs"):
        assert call(c=cache(**{null: 0})) == E_ARG
    for null in ("cu", "lengths", "table"):
        assert call(b=batch(**{null: 0})) == E_ARG
    for bad in (0, 8, 17, 24, 48, 512, -16, 2 ** 31 - 1):
        assert call(c=cache(block=bad)) == E_SHAPE
    for bad in (0, 32, 80, 96, 320, -64):
        assert call(c=cache(dim=bad)) == E_SHAPE
    for bad in (0, -1, 2 ** 31):
        assert call(c=cache(pages=bad)) == E_SHAPE
    for bad in (0, -1, 65536):
        assert call(c=cache(heads=bad)) == E_SHAPE
    for bad in (0, -1, 2 ** 20 + 1):
        assert call(b=batch(seqs=bad)) == E_SHAPE
    for bad in (0, -1, 2 ** 31 - 1):  # the last: more positions than a table may have
        assert call(b=batch(width=bad, stride=2 ** 31)) == E_SHAPE
    assert call(b=batch(stride=2)) == E_SHAPE
    for bad in (-1, 2 ** 23 + 1):
        assert call(b=batch(tokens=bad)) == E_SHAPE
    assert call(c=cache(kc=P + 8)) == E_ALIGN
    assert call(b=batch(table=P + 2)) == E_ALIGN
    assert call(dt=2) == E_DTYPE
    assert call(status=P + 1) == E_ALIGN
    assert call(b=batch(tokens=0)) == OK  # nothing to do


def test_rows():
    assert write(k=0) == E_ARG and write(v=0) == E_ARG and read(k=0) == E_ARG
    assert write(kh=63) == E_SHAPE and write(vt=-128) == E_SHAPE and write(vt=2 ** 62) == E_SHAPE
    assert write(k=P + 8) == E_ALIGN and write(vt=132) == E_ALIGN and write(kh=68) == E_ALIGN
    assert write(kt=130, dt=fp4.F32) == E_ALIGN
    assert read(v=P + 8) == E_ALIGN


def test_attention():
    assert attend(q=0) == E_ARG and attend(out=0) == E_ARG
    assert attend(heads=3) == E_SHAPE and attend(heads=0) == E_SHAPE and attend(heads=-2) == E_SHAPE
    assert attend(causal=2) == E_ARG and attend(window=-1) == E_ARG
    assert attend(window=5, causal=0) == E_ARG
    assert attend(scale=float("nan")) == E_ARG and attend(scale=float("inf")) == E_ARG
    assert attend(qh=32) == E_SHAPE and attend(qt=260) == E_ALIGN
    assert attend(out=P + 8) == E_ALIGN and attend(lse=P + 2) == E_ALIGN
    long = batch(width=1024, stride=1024)  # 16384 positions: split
    need = space(b=long)
    assert need > 0
    assert attend(b=long) == E_WORKSPACE
    assert attend(b=long, ws=P, wsb=need - 1) == E_WORKSPACE
    assert attend(b=long, ws=P + 4, wsb=need) == E_ALIGN


def test_workspace_bytes():
    assert space() == 0  # 48 positions: one split
    assert space(heads=3) == 0 and space(dt=5) == 0 and space(window=-1) == 0
    assert space(c=cache(dim=65)) == 0 and space(b=batch(tokens=0)) == 0
    # a row's partial output, reference and sum, for every split
    assert space(b=batch(width=1024, stride=1024)) % (4 * 4 * (64 + 2) * 4) == 0
    # the largest batch and table: a size or a refusal, never a small wrapped product
    huge = space(c=cache(heads=1, block=256, pages=2 ** 31 - 1),
                 b=batch(tokens=2 ** 23, seqs=1, width=2 ** 19, stride=2 ** 19), heads=65535, dt=fp4.F32)
    assert huge == 0 or huge >= 2 ** 23 * 65535 * 66 * 4


@pytest.mark.skipif(not os.path.exists(fp4_build.HIPCC), reason="hipcc not found")
@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_host_code_under_asan_ubsan(tmp_path):
    # each sanitizer flag after -Xarch_host: the GPU code is compiled without them
    san = []
    for f in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all",
              "-fno-omit-frame-pointer"):
        san += ["-Xarch_host", f]
    flags = [f for f in fp4_build.FLAGS if f != "-O3"] + ["-O1", "-g", *san]
    srcs = [os.path.join(fp4_build.CSRC, s) for s in fp4_build.SOURCES]
    srcs.append(os.path.join(ROOT, "tests", "sanitize", "kv_check.cpp"))
    objs = [str(tmp_path / (os.path.basename(s) + ".o")) for s in srcs]
    procs = [subprocess.Popen([fp4_build.HIPCC, *flags, "-c", s, "-o", o],
                              stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for s, o in zip(srcs, objs)]
    for p, s in zip(procs, srcs):
        out = p.communicate()[0]
        assert p.returncode == 0, f"hipcc failed on {s}:\n{out[-4000:]}"
    exe = str(tmp_path / "kv_check")
    subprocess.run([fp4_build.HIPCC, "--offload-arch=gfx950", *san, *objs, "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env)
    assert r.returncode == 0 and ", 0 failures" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
