"""The block-scaled product on the GPU, dense and by experts, against the definition in 64 bits."""
import pytest
import torch

import block_ref as ref
import scaled_gemm_amd as sg

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def codes(shape, g):
    """Codes of random values of every magnitude, none NaN."""
    c = torch.randint(0, 0x7F, shape, device="cuda", generator=g)
    return (c | (torch.randint(0, 2, shape, device="cuda", generator=g) << 7)).to(torch.uint8)


def scales(shape, g):
    return torch.exp(2 * torch.randn(shape, device="cuda", generator=g))


def operands(T, Ci, Co, seed, experts=None):
    g = gen(seed)
    lead = () if experts is None else (experts,)
    return (codes((T, Ci), g), scales((ref.blocks(Ci), T), g), codes(lead + (Ci, Co), g),
            scales(lead + (ref.blocks(Ci), ref.blocks(Co)), g))


def check(out, qx, sx, qw, sw):
    want, far = ref.product(qx, sx, qw, sw)
    off = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    bad = off > far
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {off.max().item()}"


# Every kernel, with whole tiles and without, sums of one block, a short block, an odd and an even
# number of them.
DENSE = [
    (1, 4096, 1024), (2, 1424, 272), (9, 1696, 1888), (16, 4112, 48),
    (1, 16, 16), (1, 128, 128), (16, 512, 528), (30, 2336, 1040), (33, 1040, 400), (65, 128, 128),
    (100, 1424, 1040), (257, 2608, 2912), (300, 944, 1680), (900, 272, 1056), (130, 400, 8000),
    (257, 1424, 3792), (900, 2112, 2128), (255, 2736, 4112), (300, 496, 8128), (257, 1808, 8128),
    (1025, 1040, 4112), (2049, 784, 4112), (4111, 272, 4240), (700, 528, 8208), (1300, 256, 4896),
    (3000, 1952, 1872), (900, 1520, 8032), (1500, 144, 16400), (1300, 128, 8656),
    (2100, 1936, 6224), (4100, 864, 7088), (1300, 240, 7888),
]


@pytest.mark.parametrize("T,Ci,Co", DENSE)
def test_dense(T, Ci, Co):
    qx, sx, qw, sw = operands(T, Ci, Co, T + Ci + Co)
    bw = sg.pack_weight_block(qw, sw)
    out = torch.full((T, Co), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert sg.gemm_block(qx, sx, bw, out=out) is out
    check(out, qx, sx, qw, sw)


KERNELS = {"block_gemm_kernel<256,256>", "block_gemm_kernel<128,256>", "block_gemm_kernel<128,128>",
           "block_gemm_kernel<64,128>", "block_gemm_kernel<64,64>", "block_gemm_kernel<32,64>",
           "block_few_kernel"}


def one_of_each():
    seen = {}
    for s in DENSE:
        seen.setdefault(sg.gemm_block_kernel(*s), s)
    return sorted(seen.values())


@pytest.mark.parametrize("T,Ci,Co", one_of_each())
def test_pitches(T, Ci, Co):
    """Slices of wider tensors: the same result, and nothing else is written."""
    qx, sx, qw, sw = operands(T, Ci, Co, 5)
    bw = sg.pack_weight_block(qw, sw)
    plain = sg.gemm_block(qx, sx, bw)
    wide = torch.full((T, Ci + 80), 0x7F, dtype=torch.uint8, device="cuda")     # NaN around them
    wide[:, 32:32 + Ci] = qx
    tall = torch.full((ref.blocks(Ci), T + 9), float("nan"), device="cuda")
    tall[:, 5:5 + T] = sx
    big = torch.full((T + 3, Co + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[:T, 8:8 + Co]
    sg.gemm_block(wide[:, 32:32 + Ci], tall[:, 5:5 + T], bw, out=out)
    assert torch.equal(out, plain)
    big[:T, 8:8 + Co] = 7.0
    assert (big == 7.0).all()


@pytest.mark.parametrize("T,Ci,Co", one_of_each())
def test_nan_codes_stay_in_their_row_and_column(T, Ci, Co):
    qx, sx, qw, sw = operands(T, Ci, Co, 6)
    qx[T // 2, Ci - 1] = 0x7F
    qw[0, Co // 3] = 0xFF
    out = sg.gemm_block(qx, sx, sg.pack_weight_block(qw, sw))
    nan = torch.isnan(out)
    assert nan[T // 2].all() and nan[:, Co // 3].all()
    assert int(nan.sum()) == T + Co - 1


@pytest.mark.parametrize("T,Ci,Co", one_of_each())
def test_infinite_scales_stay_in_their_blocks(T, Ci, Co):
    """The first block's: nothing of them in K blocks that are not there."""
    qx, sx, qw, sw = operands(T, Ci, Co, 8)
    qx, qw = (qx & 0x7F).clamp(min=8), (qw & 0x7F).clamp(min=8)      # positive codes
    sw[0, 0] = sx[0, T - 1] = float("inf")
    out = sg.gemm_block(qx, sx, sg.pack_weight_block(qw, sw)).float()
    assert (out[:, :128] == float("inf")).all() and (out[T - 1] == float("inf")).all()
    assert torch.isfinite(out[:T - 1, 128:]).all()


@pytest.mark.parametrize("T,Ci,Co", one_of_each())
def test_same_result_every_time(T, Ci, Co):
    qx, sx, qw, sw = operands(T, Ci, Co, 8)
    bw = sg.pack_weight_block(qw, sw)
    first = sg.gemm_block(qx, sx, bw)
    for _ in range(3):
        assert torch.equal(sg.gemm_block(qx, sx, bw), first)


def test_empty():
    qx = torch.empty((5, 0), dtype=torch.uint8, device="cuda")
    sx = torch.empty((0, 5), device="cuda")
    bw = sg.BlockWeight(torch.empty(0, dtype=torch.uint8, device="cuda"),
                        torch.empty((1, 0), device="cuda"), 0, 32)
    assert (sg.gemm_block(qx, sx, bw) == 0).all()
    q, s, w, c = operands(0, 128, 64, 1)
    assert sg.gemm_block(q, s, sg.pack_weight_block(w, c)).shape == (0, 64)


# ---- experts ---------------------------------------------------------------------------

def random_counts(E, R, g, kind):
    """Rows of each expert: ragged, all on one, or some without any."""
    if kind == "one":
        n = torch.zeros(E, dtype=torch.long)
        n[E // 2] = R
        return n
    p = torch.rand(E, device="cuda", generator=g).cpu() ** 3
    if kind == "holes":
        p[::2] = 0
    if float(p.sum()) == 0:
        p[0] = 1
    n = (p / p.sum() * R).long()
    n[int(p.argmax())] += R - int(n.sum())
    return n


def routing(E, T, K, g, kind, drop=0):
    """A routing of T * K pairs whose last `drop` rows belong to no expert; every token's pairs are
    anywhere, so a token may meet one expert twice."""
    R = T * K
    n = random_counts(E, R - drop, g, kind)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = n.cumsum(0)
    rows = torch.randperm(R, device="cuda", generator=g).to(torch.int32)
    slots = torch.empty(R, dtype=torch.int32, device="cuda")
    slots[rows.long()] = torch.arange(R, device="cuda", dtype=torch.int32)
    if drop:
        slots[rows[R - drop:].long()] = -1
        rows[R - drop:] = -1
    ids = torch.zeros((T, K), dtype=torch.int32, device="cuda")
    return sg.Routing(ids, torch.rand((T, K), device="cuda", generator=g), offsets.cuda(), rows,
                      slots.view(T, K))


EXPERTS = [     # experts, tokens, top_k, Ci, Co, how ragged
    (8, 1, 2, 272, 144, "ragged"), (64, 1, 6, 512, 528, "holes"), (3, 5, 1, 128, 32, "one"),
    (100, 40, 8, 400, 272, "ragged"), (16, 40, 8, 656, 400, "holes"), (8, 64, 6, 1040, 160, "ragged"),
    (5, 61, 8, 272, 528, "ragged"), (8, 333, 2, 528, 1040, "one"), (8, 333, 4, 1424, 272, "ragged"),
    (16, 700, 4, 272, 2064, "holes"), (130, 1000, 8, 144, 272, "ragged"), (4, 1500, 4, 272, 4112, "ragged"),
    (8, 4096, 2, 400, 2064, "ragged"), (512, 300, 4, 128, 144, "ragged"),
    (8, 400, 2, 144, 4112, "ragged"), (16, 700, 4, 304, 3872, "ragged"), (8, 2100, 1, 1232, 2080, "ragged"),
    (8, 700, 8, 400, 3136, "holes"), (8, 2100, 2, 1376, 2480, "ragged"), (16, 333, 8, 1184, 2768, "ragged"),
    (130, 2100, 4, 288, 1360, "ragged"), (16, 700, 1, 336, 2192, "holes"),
]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,K,Ci,Co,kind", EXPERTS)
def test_experts(E, T, K, Ci, Co, kind, gather):
    g = gen(E + T + Ci)
    r = routing(E, T, K, g, kind)
    R = T * K
    qx, sx, qw, sw = operands(T if gather else R, Ci, Co, 3 * T + Co, experts=E)
    bw = sg.pack_weight_block(qw, sw)
    out = torch.full((R, Co), float("nan"), dtype=torch.bfloat16, device="cuda")
    sg.gemm_experts(qx, sx, bw, r, gather=gather, out=out)
    at = r.offsets.tolist()
    for e in range(E):
        if at[e] < at[e + 1]:
            i = torch.arange(at[e], at[e + 1], device="cuda")
            src = r.rows[i].long() // K if gather else i
            check(out[i], qx[src], sx[:, src], qw[e], sw[e])


def one_of_each_experts():
    seen = {}
    for s in EXPERTS:
        seen.setdefault(sg.gemm_block_kernel(s[1] * s[2], s[3], s[4], experts=s[0]), s)
    return sorted(seen.values())


@pytest.mark.parametrize("E,T,K,Ci,Co,kind", one_of_each_experts())
def test_rows_of_no_expert_stay(E, T, K, Ci, Co, kind):
    """Rows past the last expert's are neither computed nor written, whatever qx holds there."""
    g = gen(9)
    drop = T
    r = routing(E, T, K, g, kind, drop=drop)
    R = T * K
    qx, sx, qw, sw = operands(R, Ci, Co, 4, experts=E)
    qx[R - drop:] = 0x7F
    sx[:, R - drop:] = float("nan")
    bw = sg.pack_weight_block(qw, sw)
    out = torch.full((R, Co), 7.0, dtype=torch.bfloat16, device="cuda")
    sg.gemm_experts(qx, sx, bw, r, out=out)
    assert (out[R - drop:] == 7.0).all()
    assert torch.isfinite(out).all() and not (out[:R - drop] == 7.0).all(1).any()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,K,Ci,Co,kind", one_of_each_experts())
def test_bad_device_values_stay_inside(E, T, K, Ci, Co, kind, gather):
    """Offsets and rows that make no sense: every access stays in the buffers (the kernels cut
    offsets to 0 .. R, and a row that names no token is one of zeros); sane experts still come out
    right."""
    g = gen(12)
    r = routing(E, T, K, g, "ragged")
    R = T * K
    qx, sx, qw, sw = operands(T if gather else R, Ci, Co, 5, experts=E)
    bw = sg.pack_weight_block(qw, sw)
    good = sg.gemm_experts(qx, sx, bw, r, gather=gather)
    guard = torch.full((R + 64, Co), 7.0, dtype=torch.bfloat16, device="cuda")
    for offsets in ([-5] * (E + 1), [1 << 30] * (E + 1), [0] + [R + 100] * E,
                    [(-1) ** e * (1 << 30) for e in range(E + 1)]):
        r.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
        sg.gemm_experts(qx, sx, bw, r, gather=gather, out=guard[32:32 + R])
        assert (guard[:32] == 7.0).all() and (guard[32 + R:] == 7.0).all()
    r = routing(E, T, K, gen(12), "ragged")
    if gather:
        assert torch.equal(r.rows, routing(E, T, K, gen(12), "ragged").rows)
        r.rows[0], r.rows[R // 2], r.rows[R - 1] = -1, R, -(1 << 31)
        out = sg.gemm_experts(qx, sx, bw, r, gather=True)
        assert (out[[0, R // 2, R - 1]] == 0).all()
        keep = torch.ones(R, dtype=torch.bool, device="cuda")
        keep[[0, R // 2, R - 1]] = False
        assert torch.equal(out[keep], good[keep])


@pytest.mark.parametrize("gather", [True, False])
def test_experts_equal_the_dense_product(gather):
    """One expert with all rows is the plain product, bit for bit: the tiled kernels add the same
    blocks in the same order whatever their tile."""
    T, Ci, Co = 777, 528, 2064
    qx, sx, qw, sw = operands(T, Ci, Co, 17)
    r = routing(1, T, 1, gen(1), "one")
    rows = torch.arange(T, device="cuda", dtype=torch.int32)
    r.rows.copy_(rows)
    a = sg.gemm_experts(qx, sx, sg.pack_weight_block(qw[None], sw[None]), r, gather=gather)
    assert torch.equal(a, sg.gemm_block(qx, sx, sg.pack_weight_block(qw, sw)))
