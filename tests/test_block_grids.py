"""Grids of the block-scaled products and weight loaders over their whole range of extents (CPU
only): a launch holds fewer than 2^32 threads, whatever the extents that a call takes."""
import os
import re
import shutil
import subprocess

import pytest

import scaled_gemm_amd as sg
from conftest import ROOT

MOST_OUTPUTS = 1 << 36


def grid_threads(T, Ci, Co):
    """Threads of the launch that a dense product of these extents makes."""
    name = sg.gemm_block_kernel(T, Ci, Co)
    if name == "block_few_kernel":
        return -(-Co // 16) * 512
    bm, bn = map(int, re.fullmatch(r"block_gemm_kernel<(\d+),(\d+)>", name).groups())
    return -(-T // bm) * -(-Co // bn) * (512 if bn == 256 else 256)


def test_dense_grids_fit_a_launch():
    rows = sorted({min(1 << 24, (1 << p) + d) for p in range(25) for d in (-1, 0, 1, 33) if (1 << p) + d > 0})
    cols = sorted({min(1 << 24, 16 * ((1 << p) + d)) for p in range(21) for d in (0, 1, 3)})
    for Ci in (0, 16, 128, 144, 8192, 1 << 17):
        for T in rows:
            for Co in cols:
                if T * Co > MOST_OUTPUTS or -(-Ci // 128) * -(-Co // 128) > 1 << 24:
                    continue
                assert grid_threads(T, Ci, Co) < 1 << 32, (T, Ci, Co)


def test_zeros_of_any_extent_are_written():
    """Without K the results are zeros: the tiles are chosen for the results alone."""
    assert sg.gemm_block_kernel(1 << 24, 0, 4096) == sg.gemm_block_kernel(1 << 24, 16, 4096)
    assert grid_threads(1 << 24, 0, 4096) < 1 << 32


def test_a_kernel_is_named_where_the_call_launches_one(monkeypatch):
    """Experts whose tiles a grid does not hold: the query and the call agree on every size."""
    monkeypatch.setenv("PTPC_FAULT", "launch")             # reports status 5 instead of launching
    seen = set()
    for E in (1, 64, 512):
        for R in (1, 100, 1 << 14, 1 << 20):
            for Co in (16, 1 << 12, 1 << 18, 1 << 19, 1 << 20, 1 << 22):
                a = 0x10000
                status = sg.lib().ptpc_gemm_experts(a, 16, a, R, a, a, a, None, 1, E, R, R, 16, Co, a, Co, None)
                assert status in (3, 5)
                assert (sg.gemm_block_kernel(R, 16, Co, experts=E) is None) == (status == 3), (E, R, Co)
                seen.add((R * Co <= MOST_OUTPUTS, status))
    assert (True, 3) in seen and (True, 5) in seen


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the ROCm headers not available")
def test_weight_grids_fit_a_launch(tmp_path):
    """The loaders' grids hold every block of the largest weight, in fewer than 2^32 threads along x."""
    src, exe = tmp_path / "grid.cpp", str(tmp_path / "grid")
    src.write_text('''#include <cstdio>
#include "block.h"
int main() {
    for (int64_t n : {int64_t(1), int64_t(5), ptpc::kWeightGridX - 1, ptpc::kWeightGridX,
                      ptpc::kWeightGridX + 1, int64_t(1) << 22, (int64_t(1) << 24) - 1, int64_t(1) << 24}) {
        const dim3 g = ptpc::weight_grid(n);
        std::printf("%lld %u %u %u\\n", (long long)n, g.x, g.y, g.z);
    }
}
''')
    subprocess.run(["g++", "-std=c++20", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I",
                    os.path.join(ROOT, "scaled_gemm_amd", "csrc"), str(src), "-o", exe], check=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")[:-1]
    assert len(lines) == 8
    for n, x, y, z in (map(int, v.split()) for v in lines):
        assert x * 256 < 1 << 32 and y <= 65535 and z == 1
        assert n <= x * y < n + x
