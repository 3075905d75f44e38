"""Block-scaled operators and experts on tensors past 2^31 and 2^32 bytes, and on weights with more
blocks than one row of a grid holds: a part far inside comes out as it does by itself, bit for bit."""
import pytest
import torch

import block_ref as ref
import scaled_gemm_amd as sg
import test_gpu_block_gemm as t

pytestmark = pytest.mark.gpu


def part(bw, e):
    """Expert e's weight as a layer of its own."""
    n = sg.packed_bytes(bw.Ci, bw.Co)
    return sg.BlockWeight(bw.data[e * n:(e + 1) * n], bw.sw[e], bw.Ci, bw.Co)


def test_quantized_experts_of_17_gb():
    """512 experts of 2064 x 15424, 17 x 121 blocks each, which are windows of one bf16 tensor."""
    E, Ci, Co, step = 512, 2064, 15424, 48
    big = torch.randn((Ci + step * (E - 1), Co), device="cuda", generator=t.gen(1)).bfloat16()
    w = big.as_strided((E, Ci, Co), (step * Co, Co, 1))
    assert E * ref.blocks(Ci) * ref.blocks(Co) > 1 << 20
    bw = sg.quant_weight_block(w)
    for e in (0, 1, 255, 256, 509, 510, 511):
        alone = sg.quant_weight_block(w[e].contiguous())
        assert torch.equal(part(bw, e).data, alone.data) and torch.equal(bw.sw[e], alone.sw)
