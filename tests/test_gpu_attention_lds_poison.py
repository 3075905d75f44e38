"""The LDS-poison debug build (libptpc_lds_poison.so) against the release build on the attention
operators, bit for bit.

In the debug build a wave that starts to refill a region of LDS -- keys and values of the tile
kernel, values of the few-row one -- overwrites it with NaN first.  The kernels keep their slots
apart with bare barriers and counted waits; a wave that read a slot after its refill had begun,
or before it had landed, would turn the rows it computes into NaN.  Every kernel runs here: both
cache types and both head sizes, tiles of 16, 32, 128 and 256 rows, odd and even numbers of key
tiles, split and whole ranges, prompts of both tile sizes.
"""
import os

import numpy as np
import pytest
import torch

import attention_ref as ref

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


def both(libs, call):
    """The call's outputs by the release and the debug build."""
    sg, release, poison = libs
    out = []
    try:
        for lib in (release, poison):
            sg._lib = lib
            out.append(call(sg))
            torch.cuda.synchronize()
    finally:
        sg._lib = release
    return out


def same(a, b):
    assert torch.isfinite(a.float()).all()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# new tokens and cached tokens of each sequence, four query heads to a key head
SHAPES = {
    "16 rows": ([1, 4, 2, 1], [1, 333, 64, 1000]),
    "32 rows": ([7, 5, 8], [200, 9, 777]),
    "16 rows, ranges": ([1, 3], [9000, 5001]),
    "two row tiles, ranges": ([14, 3], [4000, 33]),
    "128 rows": ([30, 17, 1, 25], [63, 64, 65, 500]),
    "128 rows, ranges": ([30, 20], [3000, 2050]),
    "256 rows": ([300, 70, 0, 129], [300, 130, 50, 900]),
    "256 rows, ranges": ([200, 90], [2900, 4097]),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_paged(libs, shape, D, fp8):
    print(f"attention lds poison {shape} D={D} fp8={fp8}", flush=True)
    nq, nkv = SHAPES[shape]
    Hq, Hk, page = 8, 2, 16
    rng = np.random.default_rng([D, len(shape)])
    pages, table = ref.paged_layout(rng, nkv, page)
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    draw = lambda *s: torch.randn(s, device="cuda", generator=g)          # noqa: E731
    sg = libs[0]
    cache = sg.kv_cache(pages, Hk, page, D, fp8=fp8)
    for x, d in ((cache.k, cache.dk), (cache.v, cache.dv)):
        if fp8:
            codes = draw(*x.shape).mul_(100).clamp_(-448, 448)      # beyond: NaN codes
            x.copy_(codes.to(torch.float8_e4m3fn).view(torch.uint8))
            d.fill_(0.01)
        else:
            x.copy_(draw(*x.shape))
    q = (2 * draw(sum(nq), Hq, D)).bfloat16()
    cu = i32([0] + [int(x) for x in np.cumsum(nq)])
    table, lens = table.cuda(), i32(nkv)
    a, b = both(libs, lambda sg: sg.attn_paged(q, cu, cache, table, lens, max_q=max(nq),
                                               max_kv=max(nkv)))
    same(a, b)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk,lens", [(8, 2, [77, 1, 64, 300, 129]), (128, 8, [1000, 63, 1009])])
def test_prompt(libs, D, Hq, Hk, lens):
    print(f"attention lds poison prompt Hq={Hq} D={D}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(D + Hq)
    q, k, v = (torch.randn((sum(lens), h, D), device="cuda", generator=g).bfloat16()
               for h in (Hq, Hk, Hk))
    cu = i32([0] + [int(x) for x in np.cumsum(lens)])
    a, b = both(libs, lambda sg: sg.attn_prompt(q, k, v, cu))
    same(a, b)
