"""The LDS-poison debug build (libptpc_lds_poison.so) against the release build on the block-scaled
products, bit for bit.

In the debug build a wave that refills a region of LDS overwrites it with NaN first.  The tiled
kernels keep their slots, and the parts of a slot, apart with bare barriers and counted waits; a
wave that read a part after its refill had begun, or before it had landed, would turn what it
computes into NaN.  Every kernel runs, with one to many K blocks, whole and short ones.
"""
import os

import pytest
import torch

import test_gpu_block_gemm as t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_gemm_amd as sg
    from scaled_gemm_amd import build
    assert os.path.exists(build.POISON_LIB), "build the LDS-poison variant first"
    release, path = sg.lib(), sg.LIB_PATH
    sg._lib, sg.LIB_PATH = None, build.POISON_LIB
    poison = sg.lib()
    sg._lib, sg.LIB_PATH = release, path
    return sg, release, poison


def check(libs, call):
    sg, release, poison = libs
    out = []
    try:
        for lib in (release, poison):
            sg._lib = lib
            out.append(call(sg))
            torch.cuda.synchronize()
    finally:
        sg._lib = release
    assert torch.isfinite(out[0]).all()
    assert torch.equal(*out)


@pytest.mark.parametrize("T,Ci,Co", t.DENSE)
def test_dense(libs, T, Ci, Co):
    print(f"block lds poison {T} {Ci} {Co}", flush=True)
    qx, sx, qw, sw = t.operands(T, Ci, Co, 3)
    bw = libs[0].pack_weight_block(qw, sw)
    check(libs, lambda sg: sg.gemm_block(qx, sx, bw))


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,K,Ci,Co,kind", t.EXPERTS)
def test_experts(libs, E, T, K, Ci, Co, kind, gather):
    print(f"block lds poison experts {E} {T} {K} {Ci} {Co}", flush=True)
    r = t.routing(E, T, K, t.gen(E), kind)
    qx, sx, qw, sw = t.operands(T if gather else T * K, Ci, Co, 4, experts=E)
    bw = libs[0].pack_weight_block(qw, sw)
    check(libs, lambda sg: sg.gemm_experts(qx, sx, bw, r, gather=gather))
