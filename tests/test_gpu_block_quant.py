"""Block-scaled quantization on the GPU: activations (plain and gated) and weights, against the
rule in 64 bits."""
import pytest
import torch

import block_ref as ref
import scaled_gemm_amd as sg

pytestmark = pytest.mark.gpu

# whole blocks, a short last one, fewer channels than a block; one row, odd counts, and enough
# rows that a wave takes four of them (rows * blocks >= 2^17)
SHAPES = [(1, 16), (1, 4096), (3, 128), (5, 144), (17, 272), (63, 1424), (64, 512), (333, 2736),
          (8209, 2064)]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def acts(T, C, seed, wild=True):
    g = gen(seed)
    x = torch.randn((T, C), device="cuda", generator=g)
    if wild:        # rows and channels of very different size
        x *= torch.exp(4 * torch.randn((T, 1), device="cuda", generator=g))
        x *= torch.exp(2 * torch.randn((1, C), device="cuda", generator=g))
    return x.bfloat16()


@pytest.mark.parametrize("T,C", SHAPES)
def test_plain(T, C):
    x = acts(T, C, T + C)
    if T > 2:
        x[1] = 0                                  # a row of zeros
        x[2, :min(C, 128)] = 0                    # a block of zeros
    qx, sx = sg.quant_act_block(x)
    want, scale = ref.quantized(x.double())
    assert sx.shape == (ref.blocks(C), T)
    assert torch.equal(sx.double(), scale)
    assert torch.equal(ref.values(qx), want)


def test_every_bf16_number():
    """Each finite bf16 magnitude as a block's largest, next to smaller ones of both signs: codes
    by the rule, signs of zeros included."""
    top = torch.arange(0x7F80, dtype=torch.int32, device="cuda").to(torch.int16)
    g = gen(5)
    f = torch.rand((top.numel(), 128), device="cuda", generator=g, dtype=torch.float64) * 2 - 1
    x = (top.view(torch.bfloat16).double()[:, None] * f).bfloat16()
    x[:, 7] = top.view(torch.bfloat16)
    x[:, 9] = -top.view(torch.bfloat16)
    x[:, 11] = 0.0
    x[:, 13] = -0.0
    qx, sx = sg.quant_act_block(x)
    want, scale = ref.quantized(x.double())
    assert torch.equal(sx.double(), scale)
    assert torch.equal(ref.values(qx), want)
    assert torch.equal((qx >= 128), torch.signbit(x))


@pytest.mark.parametrize("T,C", SHAPES)
def test_gated(T, C):
    """The scale is the fp32 value of silu(a) * b up to a few fp32 steps (exp 2^-23 of its own,
    the sum, the quotient, the product: within 6 half steps each of at most 2^-24, doubled for
    exp's argument), and the codes are those of the kernel's own scale except where the quotient
    lies that near to the middle between two codes."""
    x = acts(T, 2 * C, 7 * T + C, wild=False)
    x[:, :C] *= 4
    if T > 2:
        x[1, C:] = 0
        x[2] = 0
    qx, sx = sg.quant_act_block(x, gate=True)
    a, b = x[:, :C].double(), x[:, C:].double()
    h = a / (1 + torch.exp(-a)) * b
    pad = torch.zeros((T, ref.blocks(C) * 128), dtype=torch.float64, device="cuda")
    pad[:, :C] = h
    top = pad.view(T, -1, 128).abs().amax(-1).T
    want = torch.where(top == 0, torch.ones_like(top), top / 448)
    assert ((sx.double() - want).abs() <= 2.0 ** -20 * want).all()
    q = h / sx.double().T.repeat_interleave(128, 1)[:, :C]
    # any code whose range, widened by 2^-19 of it, holds the quotient
    code = ref.values(qx)
    assert (((code >= ref.e4m3(q * (1 - 2.0 ** -19))) & (code <= ref.e4m3(q * (1 + 2.0 ** -19)))) |
            ((code <= ref.e4m3(q * (1 - 2.0 ** -19))) & (code >= ref.e4m3(q * (1 + 2.0 ** -19))))).all()


def test_gated_extremes():
    """Gates far from zero, where exp overflows or vanishes, and products of the smallest numbers."""
    T, C = 9, 128
    x = torch.zeros((T, 2 * C), device="cuda", dtype=torch.bfloat16)
    x[0, :C], x[0, C:] = 1e4, 2.0                  # silu(a) = a
    x[1, :C], x[1, C:] = -1e4, 2.0                 # -0
    x[2, :C], x[2, C:] = 2.0 ** -100, 2.0 ** -40   # 2^-141: scale 2^-144
    x[3, :C], x[3, C:] = 2.0 ** -100, 2.0 ** -48   # 2^-149, the smallest fp32 number
    x[4, :C], x[4, C:] = 2.0 ** -100, 2.0 ** -60   # vanishes
    x[5, :C], x[5, C:] = 88.0, -1.0
    x[6, :C], x[6, C:] = -88.0, 1e4
    x[7, :C], x[7, C:] = 0.0, 3e38
    x[8, 0], x[8, C:] = 3.0, 3.0
    qx, sx = sg.quant_act_block(x, gate=True)
    v = ref.values(qx)
    assert torch.isfinite(sx).all() and torch.isfinite(v).all() and (sx >= 2.0 ** -144).all()
    back = v * sx[0].double()[:, None]
    a, b = x[:, :C].double(), x[:, C:].double()
    h = a / (1 + torch.exp(-a)) * b
    # a code is within half a step (2^-4), the smallest ones within 2^-10 of the scale's unit
    assert ((back - h).abs() <= 2.0 ** -4 * h.abs() * 1.001 + 2.0 ** -10 * sx[0].double()[:, None] +
            2.0 ** -149).all()
    assert (sx[0, [1, 4, 7]] == 1).all() and (v[[1, 4, 7]] == 0).all()


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("T,C,n", [(9, 272, 0), (9, 272, 5), (9, 272, 9), (9, 272, 1000),
                                   (9, 272, -3), (8209, 2064, 4100)])
def test_count(gate, T, C, n):
    """Rows from count on are left as they were, scales too; the others are the plain call's."""
    x = acts(T, 2 * C if gate else C, 3, wild=False)
    full = sg.quant_act_block(x, gate=gate)
    qx = torch.full((T, C), 0x5A, dtype=torch.uint8, device="cuda")
    sx = torch.full((ref.blocks(C), T), -7.0, device="cuda")
    count = torch.tensor([n], dtype=torch.int32, device="cuda")
    sg.quant_act_block(x, gate=gate, count=count, qx=qx, sx=sx)
    m = min(max(n, 0), T)
    assert torch.equal(qx[:m], full[0][:m]) and torch.equal(sx[:, :m], full[1][:, :m])
    assert (qx[m:] == 0x5A).all() and (sx[:, m:] == -7.0).all()


@pytest.mark.parametrize("gate", [False, True])
def test_pitches(gate):
    """Slices of wider tensors; what lies between the rows stays as it was."""
    T, C = 37, 400
    w = 2 * C if gate else C
    big = acts(T, w + 64, 11, wild=False)
    x = big[:, 16:16 + w]
    qbig = torch.full((T, C + 48), 0x5A, dtype=torch.uint8, device="cuda")
    sbig = torch.full((ref.blocks(C), T + 5), -7.0, device="cuda")
    qx, sx = qbig[:, 16:16 + C], sbig[:, 3:3 + T]
    sg.quant_act_block(x, gate=gate, qx=qx, sx=sx)
    q, s = sg.quant_act_block(x.contiguous(), gate=gate)
    assert torch.equal(qx, q) and torch.equal(sx, s)
    assert (qbig[:, :16] == 0x5A).all() and (qbig[:, 16 + C:] == 0x5A).all()
    assert (sbig[:, :3] == -7.0).all() and (sbig[:, 3 + T:] == -7.0).all()


def weight(shape, seed):
    g = gen(seed)
    w = torch.randn(shape, device="cuda", generator=g)
    return (w * torch.exp(torch.randn(shape[:-1] + (1,), device="cuda", generator=g))).bfloat16()


def unpacked(bw):
    """Codes [(experts,) Ci, Co] of a packed weight."""
    n = sg.packed_bytes(bw.Ci, bw.Co)
    parts = [sg.unpack_weight(sg.PackedWeight(bw.data[e * n:(e + 1) * n], None, bw.Ci, bw.Co))
             for e in range(bw.experts or 1)]
    return torch.stack(parts) if bw.experts else parts[0]


@pytest.mark.parametrize("shape", [(16, 16), (128, 128), (272, 144), (1424, 528), (3, 400, 272),
                                   (5, 128, 1040)])
def test_weight(shape):
    w = weight(shape, 21)
    w[..., :shape[-1] // 2] *= 100
    if shape[-2] > 128:
        w[..., :128, :16] = 0
    bw = sg.quant_weight_block(w)
    codes = unpacked(bw)
    E = shape[0] if len(shape) == 3 else 1
    Ci, Co = shape[-2:]
    sw = bw.sw.view(E, ref.blocks(Co), ref.blocks(Ci))
    for e in range(E):
        h = w.view(E, Ci, Co)[e].double()
        for b in range(ref.blocks(Ci)):
            for n in range(ref.blocks(Co)):
                k, o = slice(b * 128, (b + 1) * 128), slice(n * 128, (n + 1) * 128)
                s = ref.scale_of(h[k, o].abs().amax())
                assert sw[e, n, b].double() == s
                got = ref.values(codes.view(E, Ci, Co)[e][k, o])
                assert torch.equal(got, ref.e4m3((h[k, o] / s).float().double()))


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("shape", [(16, 16), (272, 144), (1424, 528), (3, 400, 272)])
def test_pack(shape, transposed, odd):
    """A checkpoint's codes and scales, [Ci, Co] or the transposed view of [Co, Ci], also at
    addresses that are no multiple of 16 bytes; every code, NaN included, comes through."""
    g = gen(31)
    *lead, Ci, Co = shape
    size = tuple(lead) + ((Co, Ci) if transposed else (Ci, Co))
    n = 1
    for v in size:
        n *= v
    store = torch.randint(0, 256, (n + odd,), device="cuda", generator=g).to(torch.uint8)
    codes = store[odd:].view(size)
    scales = torch.rand(tuple(lead) + (ref.blocks(Co), ref.blocks(Ci)), device="cuda", generator=g)
    scales = scales.transpose(-1, -2)
    if transposed:
        codes = codes.transpose(-1, -2)
    else:
        scales = scales.contiguous()
    bw = sg.pack_weight_block(codes, scales)
    assert torch.equal(unpacked(bw), codes)
    assert torch.equal(bw.sw, scales.transpose(-1, -2))


def test_packing_ends_with_zero_codes():
    """K bytes past Ci are zero codes (the product multiplies them)."""
    codes = torch.full((272, 32), 0x38, dtype=torch.uint8, device="cuda")
    bw = sg.pack_weight_block(codes, torch.ones((3, 1), device="cuda"))
    assert int((bw.data == 0x38).sum()) == 272 * 32 and int((bw.data != 0).sum()) == 272 * 32


def test_float8_view():
    codes = torch.randint(0, 127, (128, 128), device="cuda", generator=gen(1)).to(torch.uint8)
    s = torch.ones((1, 1), device="cuda")
    assert torch.equal(sg.pack_weight_block(codes.view(torch.float8_e4m3fn), s).data,
                       sg.pack_weight_block(codes, s).data)
