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


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


COUNTS = {0: 40, 1: 17, 200: 300, 255: 33, 256: 600, 510: 20, 511: 129}     # rows of those with any


@pytest.mark.parametrize("times", [1, 12])
@pytest.mark.parametrize("gather", [True, False])
def test_experts_whose_weights_pass_4_gb(gather, times):
    """512 experts of 2176 x 4112: each one's rows equal the product with that expert's part alone."""
    E, Ci, Co, T, K = 512, 2176, 4112, 1139 * times, 1
    g = t.gen(2)
    codes = torch.randint(0, 0x7F, (E, Ci, Co), dtype=torch.uint8, device="cuda", generator=g)
    codes ^= torch.randint(0, 2, (1, Ci, Co), dtype=torch.uint8, device="cuda", generator=g) << 7
    assert codes.numel() > 1 << 32
    sw = t.scales((E, ref.blocks(Ci), ref.blocks(Co)), g)
    bw = sg.pack_weight_block(codes, sw)
    for e in (255, 511):
        alone = sg.pack_weight_block(codes[e], sw[e])
        assert torch.equal(part(bw, e).data, alone.data) and torch.equal(bw.sw[e], alone.sw)
    del codes
    qx, sx = t.codes((T, Ci), g), t.scales((ref.blocks(Ci), T), g)
    count = torch.zeros(E, dtype=torch.long)
    for e, n in COUNTS.items():
        count[e] = n * times
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = count.cumsum(0)
    rows = torch.randperm(T, device="cuda", generator=g).to(torch.int32)
    r = sg.Routing(torch.zeros((T, K), dtype=torch.int32, device="cuda"), None, offsets.cuda(), rows, None)
    out = sg.gemm_experts(qx, sx, bw, r, gather=gather)
    for e in COUNTS:
        i = torch.arange(int(offsets[e]), int(offsets[e + 1]), device="cuda")
        src = rows[i].long() if gather else i
        assert torch.equal(out[i], sg.gemm_block(qx[src], sx[:, src].contiguous(), part(bw, e)))


def far(rows, cols, pitch, dtype):
    """A tensor [rows, cols] whose rows lie `pitch` elements apart."""
    return torch.empty((rows, pitch), dtype=dtype, device="cuda")[:, :cols]


def test_gather_over_2_gb_of_rows():
    """The most that a gather takes: 2^15 tokens 2^16 bytes apart."""
    E, T, K, Ci, Co = 8, 1 << 15, 2, 272, 528
    r = t.routing(E, T, K, t.gen(3), "ragged")
    qx, sx, qw, sw = t.operands(T, Ci, Co, 4, experts=E)
    bw = sg.pack_weight_block(qw, sw)
    wide = far(T, Ci, 1 << 16, torch.uint8)
    wide.copy_(qx)
    assert torch.equal(sg.gemm_experts(wide, sx, bw, r, gather=True),
                       sg.gemm_experts(qx, sx, bw, r, gather=True))


@pytest.mark.parametrize("T,Ci,Co", [(70001, 272, 528), (70001, 400, 48)])
def test_product_of_rows_far_apart(T, Ci, Co):
    """Rows, scales and results each over more than 2^31 bytes."""
    qx, sx, qw, sw = t.operands(T, Ci, Co, 5)
    bw = sg.pack_weight_block(qw, sw)
    q, s = far(T, Ci, 1 << 16, torch.uint8), far(ref.blocks(Ci), T, 1 << 28, torch.float32)
    out = far(T, Co, 1 << 15, torch.bfloat16)
    q.copy_(qx)
    s.copy_(sx)
    sg.gemm_block(q, s, bw, out=out)
    assert torch.equal(out, sg.gemm_block(qx, sx, bw))


@pytest.mark.parametrize("gate", [False, True])
def test_quantizer_of_rows_far_apart(gate):
    T, C = 70001, 272
    x = torch.randn((T, C * (2 if gate else 1)), device="cuda", generator=t.gen(6)).bfloat16()
    wide = far(T, x.shape[1], 1 << 16, torch.bfloat16)
    wide.copy_(x)
    q, s = far(T, C, 1 << 16, torch.uint8), far(ref.blocks(C), T, 1 << 28, torch.float32)
    sg.quant_act_block(wide, gate=gate, qx=q, sx=s)
    qx, sx = sg.quant_act_block(x, gate=gate)
    assert torch.equal(q, qx) and torch.equal(s, sx)


def test_sum_of_rows_far_apart():
    T, K, C = 10000, 4, 272
    g = t.gen(7)
    y = torch.randn((T * K, C), device="cuda", generator=g).bfloat16()
    slots = torch.randperm(T * K, device="cuda", generator=g).to(torch.int32).view(T, K)
    r = sg.Routing(slots, torch.rand((T, K), device="cuda", generator=g), None, None, slots)
    wide, out = far(T * K, C, 1 << 16, torch.bfloat16), far(T, C, 1 << 18, torch.bfloat16)
    wide.copy_(y)
    sg.combine_experts(wide, r, out=out)
    assert torch.equal(out, sg.combine_experts(y, r))


def test_routing_of_rows_far_apart():
    T, E, K = 20000, 130, 4
    x = torch.randn((T, E), device="cuda", generator=t.gen(8))
    wide = far(T, E, 1 << 16, torch.float32)
    wide.copy_(x)
    a, b = sg.route_experts(wide, K), sg.route_experts(x, K)
    for name in ("ids", "weights", "offsets", "rows", "slots"):
        assert torch.equal(getattr(a, name), getattr(b, name))
