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
RELEASE, POISON = (), ("-DPTPC_LDS_POISON",)


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

    with ThreadPoolExecutor(max_workers=4) as ex:
        return dict(ex.map(compile_one, [(f, d) for f in FILES for d in (RELEASE, POISON)]))


@pytest.mark.parametrize("name", FILES)
def test_inline_asm_touches_no_register(assembly, name):
    text = assembly[name, RELEASE]
    assert text.count("v_mfma") > 100
    bad = sorted({line for line in _asm_blocks(text) if _touches_registers(line)})
    assert not bad, bad[:5]


@pytest.mark.parametrize("name", FILES)
def test_the_debug_build_writes_its_poison(assembly, name):
    """Every attention kernel of the LDS-poison build has more 16-byte LDS writes than the
    release build's."""
    def writes(text):
        out = {}
        for m in re.finditer(r"\n(_ZN4ptpc\w*attn_(?:tile|few)_kernel\w+):", text):
            body = text[m.start():text.index(".Lfunc_end", m.start())]
            out[m.group(1)] = body.count("ds_write_b128")
        return out
    release, poison = writes(assembly[name, RELEASE]), writes(assembly[name, POISON])
    assert len(release) >= 8 and release.keys() == poison.keys()
    for k in release:
        assert poison[k] > release[k], k


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
