"""Routing, the sum over the experts, and a whole layer of experts on the GPU."""
import pytest
import torch

import block_ref as ref
import scaled_gemm_amd as sg

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def logits(T, E, seed, dtype=torch.float32):
    g = gen(seed)
    x = 2 * torch.randn((T, E), device="cuda", generator=g)
    x += torch.randn(E, device="cuda", generator=g)
    return x.to(dtype)


def check_route(r, x, k, sigmoid, bias, groups, top_groups, group_top, renorm, scale, first, local):
    ids, w = ref.route(x, k, sigmoid, bias, groups, top_groups, group_top, renorm, scale)
    assert torch.equal(r.ids.cpu(), ids)
    # rounded once to fp32; the 64-bit sums before that are off by far less
    assert ((r.weights.cpu().double() - w).abs() <= 2.0 ** -24 * w.abs() * 1.0001 + 2.0 ** -150).all()
    offsets, rows, slots = ref.layout(ids, first, local)
    assert torch.equal(r.offsets.cpu(), offsets)
    assert torch.equal(r.rows.cpu(), rows)
    assert torch.equal(r.slots.cpu(), slots)


ROUTES = [      # tokens, experts, top_k, sigmoid, bias, groups, top_groups, group_top
    (1, 1, 1, False, False, 1, 1, 2), (1, 8, 2, False, False, 1, 1, 2), (3, 60, 4, True, True, 1, 1, 2),
    (16, 256, 8, True, True, 8, 4, 2), (17, 64, 6, False, True, 8, 3, 1), (64, 160, 6, False, False, 8, 3, 1),
    (65, 128, 8, False, False, 1, 1, 2), (31, 512, 64, True, False, 64, 16, 2), (200, 65, 8, True, True, 5, 2, 2),
    (1000, 130, 3, False, True, 65 // 5, 7, 2), (2500, 512, 8, True, True, 4, 2, 2), (5, 64, 64, False, False, 1, 1, 2),
    (40, 8, 2, True, True, 8, 2, 2), (3000, 16, 1, False, False, 1, 1, 1),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,sigmoid,bias,groups,top_groups,group_top", ROUTES)
def test_route(T, E, k, sigmoid, bias, groups, top_groups, group_top, dtype):
    """bf16 logits give equal scores without a bias: then the lowest index goes first."""
    x = logits(T, E, T + E, dtype)
    b = 0.1 * torch.randn(E, device="cuda", generator=gen(1)) if bias else None
    renorm, scale = T % 2 == 0, 1.0 if T % 3 else 2.5
    r = sg.route_experts(x, k, "sigmoid" if sigmoid else "softmax", b, groups, top_groups, group_top,
                         renorm, scale)
    check_route(r, x, k, sigmoid, b, groups, top_groups, group_top, renorm, scale, 0, E)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_route_nonfinite(sigmoid, groups, top_groups):
    """Masked experts (-inf, the type's lowest), infinities, NaN, rows of nothing else."""
    inf, nan = float("inf"), float("nan")
    x = logits(12, 16, 3)
    x[0] = -inf
    x[1] = nan
    x[2, :15] = -inf
    x[3, 5] = inf
    x[4, [2, 9]] = inf
    x[5, 4] = nan
    x[6] = torch.finfo(torch.float32).min
    x[7] = 0.0
    x[8, :8] = -inf
    x[9] = -200.0
    x[10, 1], x[10, 2:] = 800.0, -800.0
    bias = torch.zeros(16, device="cuda")
    for b in (None, bias):
        r = sg.route_experts(x, 4, "sigmoid" if sigmoid else "softmax", b, groups, top_groups, 2)
        check_route(r, x, 4, sigmoid, b, groups, top_groups, 2, True, 1.0, 0, 16)
    bias[3], bias[7], bias[11] = -inf, nan, 1e30
    r = sg.route_experts(x, 4, "sigmoid" if sigmoid else "softmax", bias, groups, top_groups, 2)
    check_route(r, x, 4, sigmoid, bias, groups, top_groups, 2, True, 1.0, 0, 16)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k,groups,top_groups", [(8, 3, 1, 1), (64, 8, 1, 1), (130, 9, 1, 1), (256, 8, 8, 3),
                                                   (512, 64, 1, 1), (512, 20, 16, 4)])
def test_route_near_ties(E, k, groups, top_groups, sigmoid):
    """Scores that are equal in 32 bits, and equal or 2^-30 apart in 64."""
    x = torch.randint(0, 16, (40, E), device="cuda", generator=gen(E)).float() * 2.0 ** -30
    r = sg.route_experts(x, k, "sigmoid" if sigmoid else "softmax", None, groups, top_groups, 1)
    check_route(r, x, k, sigmoid, None, groups, top_groups, 1, True, 1.0, 0, E)


@pytest.mark.parametrize("T,first,local", [(7, 0, 4), (7, 12, 4), (50, 3, 1), (700, 5, 7), (700, 0, 16)])
def test_route_local(T, first, local):
    """The layout of some of the experts only; the others' pairs have no row."""
    x = logits(T, 16, 8)
    r = sg.route_experts(x, 3, first=first, local=local)
    check_route(r, x, 3, False, None, 1, 1, 2, True, 1.0, first, local)


def test_route_all_on_one():
    x = logits(3000, 64, 4)
    x[:, 40] += 100
    r = sg.route_experts(x, 1)
    check_route(r, x, 1, False, None, 1, 1, 2, True, 1.0, 0, 64)
    assert r.offsets[40] == 0 and r.offsets[41] == 3000


def test_route_pitch_and_empty():
    wide = logits(70, 40, 6)
    x = wide[:, 4:36]
    r = sg.route_experts(x, 2)
    check_route(r, x, 2, False, None, 1, 1, 2, True, 1.0, 0, 32)
    r = sg.route_experts(x[:0], 2)
    assert (r.offsets == 0).all() and r.offsets.shape == (33,) and r.rows.shape == (0,)


def test_route_many_tokens():
    """Chunks longer than one batch of pairs in LDS: against a sort on the GPU."""
    T, E, k = 150_000, 32, 8
    x = logits(T, E, 2)
    r = sg.route_experts(x, k)
    flat = r.ids.flatten().long()
    rows = torch.sort(flat, stable=True).indices
    assert torch.equal(r.rows.long(), rows)
    slots = torch.empty_like(rows)
    slots[rows] = torch.arange(T * k, device="cuda")
    assert torch.equal(r.slots.flatten().long(), slots)
    assert torch.equal(r.offsets.long(), torch.cat([rows.new_zeros(1),
                                                    torch.bincount(flat, minlength=E).cumsum(0)]))
    p = torch.softmax(x.double(), 1)
    assert torch.equal(r.ids.long(), p.sort(dim=1, descending=True, stable=True).indices[:, :k])


# ---- the sum -----------------------------------------------------------------------------

def check_sum(out, y, slots, weights):
    want, mag = ref.combined(y, slots, weights)
    # K fused steps of at most half a step 2^-24 of the magnitudes, then one rounding to bf16
    K = slots.shape[1]
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + K * 2.0 ** -24 * mag * 1.01 +
            2.0 ** -134).all()


@pytest.mark.parametrize("T,K,C", [(1, 1, 16), (1, 8, 4096), (5, 3, 272), (64, 6, 2048), (333, 8, 528),
                                   (33, 64, 144), (1000, 2, 1040), (7, 9, 8192), (4099, 4, 1024)])
def test_combine(T, K, C):
    g = gen(T + C)
    y = torch.randn((T * K, C), device="cuda", generator=g).bfloat16()
    slots = torch.randperm(T * K, device="cuda", generator=g).to(torch.int32).view(T, K)
    w = torch.randn((T, K), device="cuda", generator=g)
    r = sg.Routing(slots, w, None, None, slots)
    out = torch.full((T, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    check_sum(sg.combine_experts(y, r, out=out), y, slots, w)


def test_combine_without_rows():
    """Slots that name no row add nothing, not even where y or the weight is not a number."""
    T, K, C = 9, 4, 144
    g = gen(3)
    y = torch.randn((T * K, C), device="cuda", generator=g).bfloat16()
    slots = torch.arange(T * K, device="cuda", dtype=torch.int32).view(T, K).clone()
    w = torch.rand((T, K), device="cuda", generator=g)
    y[4] = float("nan")
    slots[1, 0] = -1
    slots[2] = -1
    slots[3, 1], slots[3, 2] = T * K, -(1 << 31)
    w[2] = float("nan")
    out = sg.combine_experts(y, sg.Routing(slots, w, None, None, slots))
    assert (out[2] == 0).all() and torch.isfinite(out).all()
    w[2] = 0
    check_sum(out, torch.where(torch.isnan(y), torch.zeros_like(y), y), slots, w)


def test_combine_pitches():
    T, K, C = 21, 3, 272
    g = gen(4)
    big = torch.randn((T * K, C + 40), device="cuda", generator=g).bfloat16()
    slots = torch.randperm(T * K, device="cuda", generator=g).to(torch.int32).view(T, K)
    w = torch.rand((T, K), device="cuda", generator=g)
    r = sg.Routing(slots, w, None, None, slots)
    wide = torch.full((T, C + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 8:8 + C]
    sg.combine_experts(big[:, 16:16 + C], r, out=out)
    assert torch.equal(out, sg.combine_experts(big[:, 16:16 + C].contiguous(), r))
    assert (wide[:, :8] == 7.0).all() and (wide[:, 8 + C:] == 7.0).all()


# ---- a layer of experts --------------------------------------------------------------------

def layer(x, logits, w1, w2, k, first=0, local=None, routing=None):
    """One feed-forward layer: x [T, C] bf16 -> bf16."""
    r = routing or sg.route_experts(logits, k, first=first, local=local)
    qx, sx = sg.quant_act_block(x)
    h = sg.gemm_experts(qx, sx, w1, r, gather=True)
    qh, sh = sg.quant_act_block(h, gate=True, count=r.offsets[-1:])
    return sg.combine_experts(sg.gemm_experts(qh, sh, w2, r), r), r, h


def weights(E, C, F, seed):
    g = gen(seed)
    w1 = torch.randn((E, C, 2 * F), device="cuda", generator=g) * C ** -0.5
    w2 = torch.randn((E, F, C), device="cuda", generator=g) * F ** -0.5
    return w1.bfloat16(), w2.bfloat16()


@pytest.mark.parametrize("T", [1, 5, 64, 700, 3001])
def test_layer(T):
    """The five calls one after another against the same layer in 64 bits on the dequantized
    weights.  Inputs, gated values and the two products are rounded (E4M3 2^-4 twice, bf16 2^-8
    three times); errors of a sum of many products average out: within the E4M3 half step over
    the square root of the sum's length they would be far below 2^-4 of the result's norm, which
    is the bound."""
    E, C, F, k = 16, 512, 400, 3
    w1, w2 = weights(E, C, F, 2)
    b1, b2 = sg.quant_weight_block(w1), sg.quant_weight_block(w2)
    x = torch.randn((T, C), device="cuda", generator=gen(T)).bfloat16()
    out, r, _ = layer(x, logits(T, E, T), b1, b2, k)

    def dequantized(w):
        n, ci, co = w.shape
        res = w.double()
        for b in range(0, ci, 128):
            for o in range(0, co, 128):
                blk = res[:, b:b + 128, o:o + 128]
                s = ref.scale_of(blk.abs().amax((1, 2)))[:, None, None]
                blk.copy_(ref.e4m3((blk / s).float().double()) * s)
        return res

    d1, d2 = dequantized(w1), dequantized(w2)
    want = torch.zeros((T, C), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (r.ids == e).nonzero(as_tuple=True)
        h = x[t].double() @ d1[e]
        h = torch.nn.functional.silu(h[:, :F]) * h[:, F:]
        want.index_add_(0, t, (h @ d2[e]) * r.weights[t, j].double()[:, None])
    assert (out.double() - want).norm() <= 2.0 ** -4 * want.norm()


def test_layer_over_two_gpus():
    """Experts dealt to two GPUs (here one after the other): each lays out and computes its own,
    and the sums of both add up to the layer's."""
    E, C, F, k, T = 16, 512, 400, 3, 130
    w1, w2 = weights(E, C, F, 3)
    x = torch.randn((T, C), device="cuda", generator=gen(8)).bfloat16()
    lg = logits(T, E, 9)
    whole, _, _ = layer(x, lg, sg.quant_weight_block(w1), sg.quant_weight_block(w2), k)
    parts = []
    for first in (0, 6):
        n = 6 if first == 0 else 10
        sl = slice(first, first + n)
        out, r, h = layer(x, lg, sg.quant_weight_block(w1[sl]), sg.quant_weight_block(w2[sl]), k,
                          first=first, local=n)
        parts.append(out.double())
    # each part and the whole are rounded once to bf16
    bound = 2.0 ** -8 * (parts[0].abs() + parts[1].abs() + whole.double().abs()) + 1e-6
    assert ((parts[0] + parts[1] - whole.double()).abs() <= bound).all()


def test_layer_in_a_graph():
    """The whole layer captured once and replayed on new inputs, with eager work between: every
    replay is the eager result."""
    E, C, F, k, T = 16, 512, 400, 3, 70
    b1, b2 = (sg.quant_weight_block(w) for w in weights(E, C, F, 4))
    x = torch.randn((T, C), device="cuda", generator=gen(1)).bfloat16()
    lg = logits(T, E, 1)
    for _ in range(2):
        layer(x, lg, b1, b2, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, r, _ = layer(x, lg, b1, b2, k)
    for i in range(4):
        x.copy_(torch.randn((T, C), device="cuda", generator=gen(10 + i)).bfloat16())
        lg.copy_(logits(T, E, 20 + i))
        graph.replay()
        got, rows = out.clone(), r.rows.clone()
        want, rr, _ = layer(x, lg, b1, b2, k)
        assert torch.equal(got, want) and torch.equal(rows, rr.rows)


def test_layers_on_two_streams():
    """Two layers at once on their own streams, workspaces and all: each the result it has alone."""
    E, C, F, k, T = 16, 512, 400, 3, 300
    b1, b2 = (sg.quant_weight_block(w) for w in weights(E, C, F, 5))
    xs = [torch.randn((T, C), device="cuda", generator=gen(i)).bfloat16() for i in range(2)]
    lgs = [logits(T, E, i) for i in range(2)]
    alone = [layer(x, lg, b1, b2, k)[0] for x, lg in zip(xs, lgs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(xs[i], lgs[i], b1, b2, k)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in got[i])
