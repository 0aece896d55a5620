"""The decoding layers' host code under AddressSanitizer and
UndefinedBehaviorSanitizer: tests/sanitize/layers_check.cpp with the library's sources
(the sanitizers instrument the host code only, the GPU code is never run).  No GPU is
needed."""
import os
import shutil
import subprocess

import pytest

from mxfp4_block_amax_amd import build as fp4_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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
    srcs.append(os.path.join(ROOT, "tests", "sanitize", "layers_check.cpp"))
    objs = [str(tmp_path / (os.path.basename(s) + ".o")) for s in srcs]
    procs = [subprocess.Popen([fp4_build.HIPCC, *flags, "-c", s, "-o", o],
                              stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for s, o in zip(srcs, objs)]
    for p, s in zip(procs, srcs):
        out = p.communicate()[0]
        assert p.returncode == 0, f"hipcc failed on {s}:\n{out[-4000:]}"
    exe = str(tmp_path / "layers_check")
    subprocess.run([fp4_build.HIPCC, "--offload-arch=gfx950", *san, *objs, "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env)
    assert r.returncode == 0 and ", 0 failures" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
