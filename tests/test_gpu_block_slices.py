"""The block-scaled products' kernels, each with several rows, several blocks of columns and several
K blocks: slices of wider tensors, values that must stay in their row or block, repeated calls."""
import pytest
import torch

import block_ref as ref
import scaled_gemm_amd as sg
import test_gpu_block_gemm as t

pytestmark = pytest.mark.gpu

DENSE = [   # two for each kernel where rows or K blocks differ in kind
    (9, 1696, 1888), (16, 4112, 272), (30, 2336, 1040), (33, 1040, 400), (300, 944, 1680),
    (257, 2608, 2912), (257, 1424, 3792), (900, 2112, 2128), (257, 1808, 8128), (1025, 1040, 4112),
    (900, 1520, 8032), (700, 528, 8208), (2100, 1936, 6224), (1300, 656, 7888),
]
EXPERTS = [  # experts, tokens, top_k, Ci, Co, how ragged: several K blocks each
    (100, 40, 8, 400, 272, "ragged"), (8, 333, 2, 528, 1040, "ragged"), (8, 400, 2, 144, 4112, "ragged"),
    (16, 700, 4, 272, 2064, "holes"), (8, 2100, 1, 1232, 2080, "ragged"), (8, 2100, 2, 1376, 2480, "ragged"),
]


def test_cases_reach_every_kernel_with_rows_and_blocks():
    assert {sg.gemm_block_kernel(*s) for s in DENSE} == t.KERNELS
    assert ({sg.gemm_block_kernel(T * K, Ci, Co, experts=E) for E, T, K, Ci, Co, _ in EXPERTS} ==
            t.KERNELS - {"block_few_kernel"})
    for T, Ci, Co in DENSE:
        assert T > 4 and Ci > 3 * 128 and Co > 2 * 128


def apart(qx, sx, Co, T_out):
    """The operands inside wider tensors of NaN, and an output inside a wider one of sevens."""
    T, Ci = qx.shape
    wide = torch.full((T + 2, Ci + 80), 0x7F, dtype=torch.uint8, device="cuda")
    wide[1:T + 1, 32:32 + Ci] = qx
    tall = torch.full((ref.blocks(Ci), T + 9), float("nan"), device="cuda")
    tall[:, 5:5 + T] = sx
    big = torch.full((T_out + 2, Co + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    return wide[1:T + 1, 32:32 + Ci], tall[:, 5:5 + T], big, big[1:T_out + 1, 8:8 + Co]


@pytest.mark.parametrize("T,Ci,Co", DENSE)
def test_pitches(T, Ci, Co):
    qx, sx, qw, sw = t.operands(T, Ci, Co, 5)
    bw = sg.pack_weight_block(qw, sw)
    q, s, big, out = apart(qx, sx, Co, T)
    sg.gemm_block(q, s, bw, out=out)
    assert torch.equal(out, sg.gemm_block(qx, sx, bw))
    t.check(out, qx, sx, qw, sw)
    out[:] = 7.0
    assert (big == 7.0).all()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,K,Ci,Co,kind", EXPERTS)
def test_expert_pitches(E, T, K, Ci, Co, kind, gather):
    """ldq, lds and ldo of the experts' products, gathered and in order."""
    r = t.routing(E, T, K, t.gen(E + Ci), kind)
    qx, sx, qw, sw = t.operands(T if gather else T * K, Ci, Co, 6, experts=E)
    bw = sg.pack_weight_block(qw, sw)
    q, s, big, out = apart(qx, sx, Co, T * K)
    sg.gemm_experts(q, s, bw, r, gather=gather, out=out)
    assert torch.equal(out, sg.gemm_experts(qx, sx, bw, r, gather=gather))
    at = r.offsets.tolist()
    for e in range(E):
        if at[e] < at[e + 1]:
            i = torch.arange(at[e], at[e + 1], device="cuda")
            src = r.rows[i].long() // K if gather else i
            t.check(out[i], qx[src], sx[:, src], qw[e], sw[e])
    out[:] = 7.0
    assert (big == 7.0).all()


@pytest.mark.parametrize("T,Ci,Co", DENSE)
def test_nan_codes_stay_in_their_row_and_column(T, Ci, Co):
    qx, sx, qw, sw = t.operands(T, Ci, Co, 6)
    qx[T // 2, Ci - 1] = 0x7F
    qw[0, Co // 3] = 0xFF
    nan = torch.isnan(sg.gemm_block(qx, sx, sg.pack_weight_block(qw, sw)))
    assert nan[T // 2].all() and nan[:, Co // 3].all()
    assert int(nan.sum()) == T + Co - 1 < T * Co // 4


@pytest.mark.parametrize("T,Ci,Co", DENSE)
def test_infinite_scales_stay_in_their_rows_and_blocks(T, Ci, Co):
    """Of a middle row and a middle block of columns, in the first and in the last K block."""
    qx, sx, qw, sw = t.operands(T, Ci, Co, 8)
    qx, qw = (qx & 0x7F).clamp(8, 0x7E), (qw & 0x7F).clamp(8, 0x7E)      # positive, none NaN
    sw[0, 1] = sx[ref.blocks(Ci) - 1, T // 2] = float("inf")
    out = sg.gemm_block(qx, sx, sg.pack_weight_block(qw, sw)).float()
    inf = torch.zeros((T, Co), dtype=torch.bool, device="cuda")
    inf[:, 128:256] = True
    inf[T // 2] = True
    assert inf.any() and not inf.all()
    assert (out[inf] == float("inf")).all() and torch.isfinite(out[~inf]).all()


@pytest.mark.parametrize("T,Ci,Co", DENSE)
def test_same_result_every_time(T, Ci, Co):
    qx, sx, qw, sw = t.operands(T, Ci, Co, 9)
    bw = sg.pack_weight_block(qw, sw)
    first = sg.gemm_block(qx, sx, bw)
    for _ in range(5):
        assert torch.equal(sg.gemm_block(qx, sx, bw), first)


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,T,K,Ci,Co,kind", EXPERTS)
def test_same_result_of_experts_every_time(E, T, K, Ci, Co, kind, gather):
    r = t.routing(E, T, K, t.gen(E + Ci), kind)
    qx, sx, qw, sw = t.operands(T if gather else T * K, Ci, Co, 6, experts=E)
    bw = sg.pack_weight_block(qw, sw)
    out = [sg.gemm_experts(qx, sx, bw, r, gather=gather) for _ in range(5)]
    at = int(r.offsets[-1])
    assert all(torch.equal(o[:at], out[0][:at]) for o in out[1:])
