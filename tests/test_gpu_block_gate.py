"""The gated quantizer at the ends of its range, each row measured against the formula and not
against the kernel's own scale.

silu(a) * b in fp32 is a / (1 + exp(-a)) * b.  The kernel's steps: exp(-a) within 2^-22 (its
instruction 2^-23, what the argument lost and the product with it 2^-24 each), the sum 2^-24, the
reciprocal 2^-23, two products 2^-24 each: 9 * 2^-24, and 2^-24 more for the scale's quotient; in
all less than 2^-20, and a product that is no longer a normal number is off by at most a step,
2^-149."""
import pytest
import torch

import block_ref as ref
import scaled_gemm_amd as sg

pytestmark = pytest.mark.gpu


def formula(a, b):
    """In 64 bits, on the CPU; zero where exp(-a) overflows fp32, as the fp32 formula has it."""
    a, b = a.double().cpu(), b.double().cpu()
    h = a / (1 + torch.exp(-a)) * b
    return torch.where(torch.exp(-a) < 2.0 ** 128, h, torch.zeros_like(h))


def check(x, C):
    qx, sx = sg.quant_act_block(x, gate=True)
    h = formula(x[:, :C], x[:, C:])
    top = h.abs().view(h.shape[0], -1, 128).amax(-1)
    sx = sx.T.double().cpu()
    want = (top / 448).clamp_min(2.0 ** -144)
    want = torch.where(top < 2.0 ** -150, torch.ones_like(want), want)
    assert ((sx - want).abs() <= 2.0 ** -20 * want + 2.0 ** -149).all()
    low = (top >= 2.0 ** -149) & (top / 448 * (1 + 2.0 ** -19) < 2.0 ** -145)
    assert (sx[low] == 2.0 ** -144).all()
    s = sx.repeat_interleave(128, 1)
    q, off = h / s, (h / s).abs() * 2.0 ** -19 + 2.0 ** -149 / s
    code = ref.values(qx).cpu()
    assert ((code >= ref.e4m3(q - off)) & (code <= ref.e4m3(q + off))).all()
    return qx.cpu(), sx, h, low


def halves(T, C):
    x = torch.zeros((T, 2 * C), device="cuda", dtype=torch.bfloat16)
    return x, x[:, :C], x[:, C:]


@pytest.mark.parametrize("b", [1e4, -3e30, 1.0])
def test_every_gate_whose_exponential_is_large(b):
    """-80 to -95 in bf16's steps of a half.  From -87.5 to -88.5 1 + exp(88) lies above 2^126 and its
    reciprocal below the normal numbers; from -89 on it has overflowed, and the product is -0."""
    gates = torch.arange(-95, -80, 0.5)
    x, a, u = halves(len(gates), 256)
    a[:], u[:] = gates[:, None], b
    qx, sx, h, _ = check(x, 256)
    there = gates >= -88.5
    assert (h[there] != 0).all() and (qx[there] == (0xFE if b > 0 else 0x7E)).all()
    assert (sx[there] < 1).all() and (sx[~there] == 1).all() and (qx[~there] & 0x7F == 0).all()


def test_gates_of_both_ends_in_one_block():
    x, a, u = halves(64, 128)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    a[:] = torch.rand(a.shape, device="cuda", generator=g) * 200 - 100
    u[:] = torch.randn(u.shape, device="cuda", generator=g)
    u[32:] *= torch.where(a[32:] < 0, 1e30, 1e-6).bfloat16()
    check(x, 128)


def test_products_of_the_smallest_numbers():
    """Products from 2^-127 down to below 2^-149 (the gate's half is exact there): the scale stops at
    2^-144, and codes say what is left."""
    x, a, u = halves(300, 128)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    a[:] = torch.exp2(torch.rand(a.shape, device="cuda", generator=g) - 100)
    u[:] = torch.exp2(torch.rand(u.shape, device="cuda", generator=g) - 27)
    u *= torch.where(torch.rand(u.shape, device="cuda", generator=g) < 0.5, -1.0, 1.0).bfloat16()
    u *= torch.exp2(-torch.arange(300, device="cuda") / 10.0)[:, None].bfloat16()
    a[:, 1], u[:, 0] = 0, 0
    qx, sx, h, low = check(x, 128)
    assert int(low.sum()) > 30
    # 2^-141 and the smallest number itself, by hand
    x, a, u = halves(2, 128)
    a[:], u[0], u[1] = 2.0 ** -100, 2.0 ** -40, 2.0 ** -48
    qx, sx, _, low = check(x, 128)
    assert low.all() and (ref.values(qx[0]) == 8.0).all() and (ref.values(qx[1]) == 2.0 ** -5).all()
