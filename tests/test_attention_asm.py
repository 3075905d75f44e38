"""Static check of the attention kernels' gfx950 assembly (no GPU needed).

Between an MFMA and the vector instruction that reads its result the hardware wants wait
states, which the compiler inserts for instructions that it made itself and not for inline
asm.  The attention kernels' MFMAs are builtins, so all that is asked of their inline asm is
that it touches no register: this test compiles both files and looks into every asm block.
"""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from conftest import ROOT

HIPCC = "/opt/rocm/bin/hipcc"
CSRC = os.path.join(ROOT, "scaled_gemm_amd", "csrc")
FILES = ["attn_tile.hip", "attn_few.hip"]


def _asm_blocks(text):
    """Instructions of every inline-asm block of an assembly file."""
    for m in re.finditer(r";;#ASMSTART\n(.*?);;#ASMEND", text, re.S):
        for line in m.group(1).split("\n"):
            line = line.split(";")[0].strip()
            if line:
                yield line


def _touches_registers(line):
    return re.search(r"\b[av](\d+\b|\[\d+:\d+\])", line) is not None


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("attn_asm")

    def compile_one(name):
        out = d / (name + ".s")
        subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++20", "-ffp-contract=off",
                        "-fno-gpu-rdc", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                        "--cuda-device-only", "-S", "-x", "hip", os.path.join(CSRC, name),
                        "-o", str(out)], check=True, capture_output=True, timeout=600)
        return name, out.read_text()

    with ThreadPoolExecutor(max_workers=2) as ex:
        return dict(ex.map(compile_one, FILES))


@pytest.mark.parametrize("name", FILES)
def test_inline_asm_touches_no_register(assembly, name):
    text = assembly[name]
    assert text.count("v_mfma") > 100
    bad = sorted({line for line in _asm_blocks(text) if _touches_registers(line)})
    assert not bad, bad[:5]


def test_the_scan_finds_a_reader():
    """The scan itself: a vector instruction in an asm block is found, outside it is not."""
    block = "\t;;#ASMSTART\n\t{}\n\t;;#ASMEND\n"
    found = lambda line: [_touches_registers(x) for x in _asm_blocks(block.format(line))]  # noqa: E731
    assert found("v_max3_f32 v1, v2, v3, v4") == [True]
    assert found("v_accvgpr_read_b32 v1, a2") == [True]
    assert found("ds_read_b128 v[4:7], v1") == [True]
    assert found("s_barrier") == [False]
    assert found("s_waitcnt vmcnt(0) ; v3") == [False]
    assert not list(_asm_blocks("\tv_max3_f32 v1, v2, v3, v4\n"))
