"""Every kernel with matrix instructions waits for them, along every way through its
code.  Compiles the library's sources to assembly; no GPU is needed."""
import os
import subprocess

import pytest

from mxfp4_block_amax_amd import build as fp4_build
from tests import _waits

SOURCES = ["fp4_gemm.hip", "fp4_linear.hip", "fp4_moe.hip", "fp4_attention.hip"]
MFMA = "v_mfma_f32_16x16x32_bf16 v[6:9], v[0:3], v[10:13], "


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    folder = tmp_path_factory.mktemp("assembly")
    flags = [f for f in fp4_build.FLAGS if f != "-fPIC"]
    running = {}
    for source in SOURCES:
        out = str(folder / source.replace(".hip", ".s"))
        running[source] = out, subprocess.Popen(
            [fp4_build.HIPCC, *flags, "-S", "--cuda-device-only",
             os.path.join(fp4_build.CSRC, source), "-o", out],
            stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    texts = {}
    for source, (out, process) in running.items():
        said = process.communicate()[0]
        assert process.returncode == 0, f"hipcc failed on {source}:\n{said[-4000:]}"
        with open(out) as f:
            texts[source] = f.read()
    return texts


@pytest.mark.skipif(not os.path.exists(fp4_build.HIPCC), reason="hipcc not found")
@pytest.mark.parametrize("source", SOURCES)
def test_kernels_wait(assembly, source):
    kernels = _waits.functions(assembly[source])
    assert sum(any(op.startswith("v_mfma") for op, _ in code) for code in kernels.values()) >= 4
    early = {name: sorted(found) for name, code in kernels.items()
             if (found := _waits.too_early(code))}
    assert not early, early


@pytest.mark.parametrize("code,early", [
    (MFMA + "0\ns_nop 7\nv_add_f32 v1, v6, v6", False),
    (MFMA + "0\ns_nop 6\nv_add_f32 v1, v6, v6", True),
    (MFMA + "0\nds_write_b32 v1, v9", True),
    (MFMA + "0\nv_mfma_f32_16x16x32_bf16 v[6:9], v[0:3], v[10:13], v[6:9]\ns_nop 7\nv_mov_b32 v1, v6",
     False),
    (MFMA + "0\nv_mfma_f32_16x16x32_bf16 v[20:23], v[6:9], v[10:13], 0", True),
    # a shorter way around what waits
    (MFMA + "0\ns_cbranch_vccz .LBB0_1\ns_nop 7\n.LBB0_1:\nv_mov_b32 v1, v6", True),
    (MFMA + "v[20:23]\ns_nop 1\nv_mov_b32 v20, v1", True),
    (MFMA + "v[20:23]\ns_nop 2\nv_mov_b32 v20, v1", False)])
def test_what_is_looked_for(code, early):
    (found,) = _waits.functions("_Zkernel:\n" + code + "\ns_endpgm").values()
    assert bool(_waits.too_early(found)) == early
