"""The GPU tests of the block-scaled products reach every kernel the host can choose (CPU only)."""
import scaled_gemm_amd as sg
import test_gpu_block_gemm as t


def test_choice_is_a_known_kernel():
    seen = {sg.gemm_block_kernel(T, Ci, Co) for T in (1, 7, 16, 17, 64, 100, 256, 400, 1000, 4096, 20000)
            for Ci in (0, 16, 1024, 8192, 1 << 17) for Co in (16, 272, 2048, 4112, 8192, 28672)}
    assert seen == t.KERNELS
    seen = {sg.gemm_block_kernel(R, Ci, Co, experts=E) for R in (1, 50, 700, 5000, 100000)
            for E in (1, 8, 60, 512) for Ci in (16, 2048) for Co in (16, 1408, 4096)}
    assert seen == t.KERNELS - {"block_few_kernel"}


def test_cases_reach_every_kernel():
    assert {sg.gemm_block_kernel(*s) for s in t.DENSE} == t.KERNELS
    assert ({sg.gemm_block_kernel(T * K, Ci, Co, experts=E) for E, T, K, Ci, Co, _ in t.EXPERTS} ==
            t.KERNELS - {"block_few_kernel"})


def test_queries_reject_what_the_calls_reject():
    assert sg.gemm_block_kernel(0, 256, 512) is None
    assert sg.gemm_block_kernel(16, 8, 512) is None
    assert sg.gemm_block_kernel(16, 256, 520) is None
    assert sg.gemm_block_kernel(16, (1 << 17) + 16, 512) is None
    assert sg.gemm_block_kernel(16, 256, 512, experts=513) is None
