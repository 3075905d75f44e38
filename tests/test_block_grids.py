"""Grids of the block-scaled products over their whole range of extents (CPU only): a launch holds
fewer than 2^32 threads, whatever the extents that a call takes."""
import re

import scaled_gemm_amd as sg

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


def test_no_kernel_is_named_for_experts_that_are_refused():
    """More tiles than a grid holds: the query says so, as the call does."""
    assert sg.gemm_block_kernel(1 << 14, 16, 1 << 22, experts=512) is None
    assert sg.gemm_block_kernel(1 << 14, 16, 1 << 20, experts=512) is not None
    assert sg.gemm_block_kernel(1 << 14, 16, 1 << 22) is not None
