"""Static checks of the block-scaled kernels' gfx950 assembly (no GPU needed).

Their MFMAs are builtins, for which the compiler keeps the wait states between an MFMA and what
reads its result; so their inline asm must touch no register.  No kernel spills, and the tiled
ones keep their sums in plain registers (the fused multiply-adds cannot reach the others).
"""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from conftest import ROOT

HIPCC = "/opt/rocm/bin/hipcc"
CSRC = os.path.join(ROOT, "scaled_gemm_amd", "csrc")
FILES = ["block_gemm.hip", "block_few.hip", "block_quant.hip", "experts.hip"]


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("block_asm")

    def compile_one(item):
        name, defines = item
        out = d / (name + "".join(defines) + ".s")
        subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++20", "-ffp-contract=off",
                        "-fno-gpu-rdc", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", *defines, "-I", os.path.join(ROOT, "include"),
                        "-I", CSRC, "--cuda-device-only", "-S", "-x", "hip",
                        os.path.join(CSRC, name), "-o", str(out)],
                       check=True, capture_output=True, timeout=600)
        return item, out.read_text()

    items = [(f, ()) for f in FILES] + [("block_gemm.hip", ("-DPTPC_LDS_POISON",))]
    with ThreadPoolExecutor(max_workers=5) as ex:
        return dict(ex.map(compile_one, items))


@pytest.mark.parametrize("name", FILES)
def test_inline_asm_touches_no_register(assembly, name):
    text = assembly[name, ()]
    for m in re.finditer(r";;#ASMSTART\n(.*?);;#ASMEND", text, re.S):
        for line in m.group(1).split("\n"):
            line = line.split(";")[0].strip()
            assert not re.search(r"\b[av](\d+\b|\[\d+:\d+\])", line), line


@pytest.mark.parametrize("name", FILES)
def test_no_kernel_spills(assembly, name):
    text = assembly[name, ()]
    kernels = re.findall(r"\.amdhsa_kernel (\S+)", text)
    assert kernels
    assert not re.search(r"scratch_(load|store)", text)
    assert "v_pk_fma_f32" not in text and "v_pk_mul_f32" not in text and "v_pk_add_f32" not in text
    if name == "block_gemm.hip":
        assert len(kernels) == 12 and "v_accvgpr" not in text


def test_the_debug_build_writes_its_poison(assembly):
    def writes(text):
        return {m.group(1): text[m.start():text.index(".Lfunc_end", m.start())].count("ds_write_b128")
                for m in re.finditer(r"\n(_ZN4ptpc\w*block_gemm_kernel\w+):", text)}
    release = writes(assembly["block_gemm.hip", ()])
    poison = writes(assembly["block_gemm.hip", ("-DPTPC_LDS_POISON",)])
    assert len(release) == 12 and release.keys() == poison.keys()
    for k in release:
        assert poison[k] > release[k], k
