"""Corners of the attention operators on the GPU: tiny heads, scales of any sign, and values
that are not finite where some rows see them and others do not."""
import numpy as np
import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_gemm_amd
    scaled_gemm_amd.lib()
    return scaled_gemm_amd


def note(msg):
    print(msg, flush=True)


def bf16(rng, *shape, gain=1.0):
    return torch.from_numpy((gain * rng.standard_normal(shape)).astype(np.float32)).bfloat16()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [0, 3, 8, 12, 16])
def test_tiny_keys_stay_numbers(sg, D, power):
    """Keys near the smallest fp32 numbers: bf16 subnormals, rotated by a table whose cosines are
    2^-power.  amax / 448 then has few bits left, or none.  A cached value is within its E4M3
    step (2^-4 of it, or half the smallest step of 2^-9 scales) of the rotated one."""
    note(f"tiny keys D={D} power={power}")
    rng = np.random.default_rng([D, power])
    T, H = 12, 2
    bits = torch.from_numpy(rng.integers(1, 6, (T, H, D)).astype(np.int16))     # n * 2^-133
    k = bits.view(torch.bfloat16)
    k[3, 0] = 0
    v = bf16(rng, T, H, D)
    table = torch.zeros((1, D))
    table[:, :D // 2] = 2.0 ** -power
    cache = sg.kv_cache(1, H, 16, D, fp8=True)
    sg.rope_append(k[:, :0].cuda(), k.cuda(), v.cuda(), table.cuda(),
                   torch.zeros(T, dtype=torch.int32).cuda(), torch.arange(T).cuda(), cache)
    codes = ref.e4m3_values(cache.k.cpu())[0, :, :T].transpose(0, 1)
    scale = cache.dk.cpu().double()[0, :, :T].transpose(0, 1)[..., None]
    assert torch.isfinite(codes).all() and torch.isfinite(scale).all()
    want = k.double() * 2.0 ** -power
    want = (want / 2.0 ** -149).round() * 2.0 ** -149       # the rotation's fp32 product
    off = (codes * scale - want).abs()
    assert (off <= 1.01 * want.abs() * 2.0 ** -4 + scale * 2.0 ** -10).all()
    assert (scale[3, 0] == 1).all()
