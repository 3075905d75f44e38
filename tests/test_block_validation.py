"""Refusals of the block-scaled operators and the experts (CPU only): the C ABI before any HIP
call, and the Python binding before any call of the library; the GPU and stream of each call."""
import os
import shutil
import subprocess
from contextlib import nullcontext
from types import SimpleNamespace

import pytest
import torch

import scaled_gemm_amd as sg
from conftest import ROOT

OK, NULLP, SHAPE, UNSUPPORTED, ALIGN, HIP = range(6)
A, B, C, D, E, F, G = (0x10000 * i for i in range(1, 8))      # never dereferenced
MIS = 0x10008


@pytest.fixture
def no_launch(monkeypatch):
    """Whatever passes validation reports PTPC_ERR_HIP instead of launching."""
    monkeypatch.setenv("PTPC_FAULT", "launch")


def quant(**kw):
    a = dict(x=A, T=3, Ci=272, ldx=544, gate=1, count=B, qx=C, ldq=272, sx=D, lds=3)
    a.update(kw)
    return sg.lib().ptpc_quant_act_block(*a.values(), None)


def test_quant_refusals(no_launch):
    assert quant() == HIP and quant(count=None) == HIP and quant(gate=0, ldx=272) == HIP
    assert quant(T=0) == OK and quant(Ci=0) == OK
    for bad in (dict(T=-1), dict(Ci=-16), dict(ldx=536), dict(ldx=264, gate=0), dict(ldq=256),
                dict(lds=2)):
        assert quant(**bad) == SHAPE, bad
    for bad in (dict(Ci=264), dict(T=(1 << 24) + 1, lds=1 << 25), dict(ldx=(1 << 22) + 8),
                dict(ldq=(1 << 22) + 16), dict(lds=(1 << 28) + 1)):
        assert quant(**bad) == UNSUPPORTED, bad
    for k in ("x", "qx", "sx"):
        assert quant(**{k: None}) == NULLP, k
    for bad in (dict(x=MIS), dict(qx=MIS), dict(sx=MIS + 2), dict(count=MIS + 1), dict(ldx=548),
                dict(ldq=280)):
        assert quant(**bad) == ALIGN, bad


def weight(**kw):
    a = dict(w=A, E=4, Ci=272, Co=400, ldw=400, we=400 * 272, packed=B, sw=C)
    a.update(kw)
    return sg.lib().ptpc_quant_weight_block(*a.values(), None)


def pack(**kw):
    a = dict(codes=A + 1, ce=400 * 272, ck=400, co=1, scales=B, se=12, sk=4, so=1, E=4, Ci=272,
             Co=400, packed=C, sw=D)
    a.update(kw)
    return sg.lib().ptpc_pack_weight_block(*a.values(), None)


def test_weight_refusals(no_launch):
    for f in (weight, pack):
        assert f() == HIP and f(E=0) == OK and f(Co=0) == OK and f(Ci=0) == OK
        for bad in (dict(E=-1), dict(Ci=-1), dict(Co=-1)):
            assert f(**bad) == SHAPE, bad
        for bad in (dict(E=513), dict(Ci=264), dict(Co=392), dict(Ci=(1 << 17) + 16),
                    dict(E=512, Ci=1 << 17, Co=16 * 128 * 16 + 16, **(dict(ldw=1 << 20) if f is weight else {}))):
            assert f(**bad) == UNSUPPORTED, bad
        assert f(packed=None) == NULLP and f(sw=None) == NULLP
        assert f(packed=MIS) == ALIGN and f(sw=MIS + 2) == ALIGN
    assert weight(ldw=392) == SHAPE and weight(we=-8) == SHAPE and weight(w=None) == NULLP
    assert weight(ldw=(1 << 22) + 8) == UNSUPPORTED
    assert weight(w=MIS) == ALIGN and weight(ldw=404) == ALIGN and weight(we=404) == ALIGN
    assert weight(E=1, we=404) == HIP                       # one weight: its stride says nothing
    assert pack(ck=1, co=272) == HIP and pack(ck=-1) == SHAPE and pack(so=-1) == SHAPE
    assert pack(ck=400, co=2) == UNSUPPORTED and pack(codes=None) == NULLP
    assert pack(scales=None) == NULLP and pack(scales=MIS + 1) == ALIGN


def dense(**kw):
    a = dict(qx=A, ldq=272, sx=B, lds=5, wp=C, sw=D, T=5, Ci=272, Co=400, out=E, ldo=400)
    a.update(kw)
    return sg.lib().ptpc_gemm_block(*a.values(), None)


def experts(**kw):
    a = dict(qx=A, ldq=272, sx=B, lds=10, wp=C, sw=D, off=F, rows=G, k=2, E=4, T=5, R=10, Ci=272,
             Co=400, out=E, ldo=400)
    a.update(kw)
    return sg.lib().ptpc_gemm_experts(*a.values(), None)


def test_product_refusals(no_launch):
    for f in (dense, experts):
        assert f() == HIP and f(Co=0) == OK and f(Ci=0, ldq=0, qx=None, sx=None, wp=None) == HIP
        for bad in (dict(T=-1), dict(Ci=-1), dict(ldq=256), dict(ldo=392), dict(lds=4)):
            assert f(**bad) == SHAPE, bad
        for bad in (dict(Ci=264), dict(Co=392), dict(ldq=(1 << 22) + 16), dict(ldo=(1 << 22) + 8),
                    dict(lds=(1 << 28) + 1)):
            assert f(**bad) == UNSUPPORTED, bad
        for k in ("qx", "sx", "wp", "sw", "out"):
            assert f(**{k: None}) == NULLP, k
        for bad in (dict(qx=MIS), dict(wp=MIS), dict(out=MIS), dict(sx=MIS + 2), dict(sw=MIS + 1),
                    dict(ldq=280), dict(ldo=404)):
            assert f(**bad) == ALIGN, bad
    assert dense(T=0, lds=0) == OK
    assert dense(T=1 << 24, lds=1 << 24, Co=1 << 13, ldo=1 << 13) == UNSUPPORTED     # outputs
    assert experts(R=0) == OK and experts(E=0) == OK and experts(off=None) == NULLP
    assert experts(off=MIS + 2) == ALIGN and experts(rows=MIS + 2) == ALIGN
    assert experts(rows=None) == SHAPE and experts(rows=None, T=10) == HIP
    assert experts(k=0) == UNSUPPORTED and experts(k=65) == UNSUPPORTED
    assert experts(E=513) == UNSUPPORTED and experts(R=-1) == SHAPE
    # rows of a gather beyond one 32-bit offset
    assert experts(T=1 << 20, lds=1 << 20, ldq=2048) == HIP
    assert experts(T=(1 << 20) + 1, lds=1 << 21, ldq=2048) == UNSUPPORTED
    # more tiles than a grid holds
    assert experts(E=512, R=1 << 14, Ci=16, ldq=16, Co=1 << 22, ldo=1 << 22) == UNSUPPORTED


def route(**kw):
    a = dict(logits=A, bf16=0, ldl=64, bias=B, T=100, E=64, k=6, sigmoid=1, groups=8, top_groups=3,
             group_top=2, renorm=1, scale=1.0, first=0, local=64, ids=C, w=D, off=E, rows=F, slots=G,
             ws=A, nbytes=1 << 20)
    a.update(kw)
    return sg.lib().ptpc_route_experts(*a.values(), None)


def test_route_refusals(no_launch):
    assert route() == HIP and route(bias=None) == HIP and route(bf16=1, logits=A + 2) == HIP
    assert route(T=0, logits=None, ids=None, w=None, rows=None, slots=None) == HIP     # offsets
    assert route(first=60, local=4) == HIP
    for bad in (dict(T=-1), dict(E=-1), dict(k=-1), dict(ldl=63), dict(groups=0), dict(top_groups=0),
                dict(top_groups=9), dict(first=-1), dict(local=-1), dict(first=1), dict(first=65),
                dict(nbytes=100)):
        assert route(**bad) == SHAPE, bad
    for bad in (dict(E=0, local=0), dict(E=513, ldl=513), dict(k=0), dict(k=65, groups=1, top_groups=1),
                dict(k=25), dict(groups=7), dict(groups=128, top_groups=1, E=128, ldl=128), dict(group_top=0),
                dict(group_top=3), dict(local=0), dict(ldl=(1 << 22) + 1), dict(T=1 << 26)):
        assert route(**bad) == UNSUPPORTED, bad
    for k in ("logits", "ids", "w", "off", "rows", "slots", "ws"):
        assert route(**{k: None}) == NULLP, k
    for bad in (dict(logits=A + 2), dict(logits=A + 1, bf16=1), dict(bias=MIS + 2), dict(ids=MIS + 1),
                dict(off=MIS + 2), dict(ws=MIS)):
        assert route(**bad) == ALIGN, bad


def test_route_workspace():
    f = sg.route_experts_workspace_bytes
    assert f(0, 64) == 0 and f(1, 64) == 0 and f(16, 64) == 0
    assert f(17, 64) == 2 * 64 * 4 and f(1 << 20, 512) <= 256 * 512 * 4 and f(-1, 4) == 0
    assert f(100, 0) == 0 and f(100, 513) == 0


def combine(**kw):
    a = dict(y=A, ldy=272, R=10, slots=B, w=C, T=5, k=2, C=272, out=D, ldo=272)
    a.update(kw)
    return sg.lib().ptpc_combine_experts(*a.values(), None)


def test_combine_refusals(no_launch):
    assert combine() == HIP and combine(T=0) == OK and combine(C=0) == OK
    assert combine(R=0, y=None) == HIP
    for bad in (dict(T=-1), dict(R=-1), dict(k=-1), dict(C=-1), dict(ldy=256), dict(ldo=256)):
        assert combine(**bad) == SHAPE, bad
    for bad in (dict(C=264), dict(k=0), dict(k=65), dict(T=1 << 28), dict(ldy=(1 << 22) + 8)):
        assert combine(**bad) == UNSUPPORTED, bad
    for k in ("y", "slots", "w", "out"):
        assert combine(**{k: None}) == NULLP, k
    for bad in (dict(y=MIS), dict(out=MIS), dict(slots=MIS + 2), dict(w=MIS + 1), dict(ldy=276),
                dict(ldo=276)):
        assert combine(**bad) == ALIGN, bad


# ---- the binding ----------------------------------------------------------------------------

class Library:
    """Size queries by the real library; every other call notes the current GPU and its stream."""

    def __init__(self, real, state):
        self.real, self.state = real, state

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*a):
            self.state.calls.append((name, self.state.current, a[-1]))
            self.state.args = a
            return self.state.status
        call.__name__ = name
        return call


@pytest.fixture
def gpus(monkeypatch):
    """CPU tensors are those of GPU -1, GPU 0 is current."""
    state = SimpleNamespace(current=0, calls=[], status=0, args=None)

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, state.current = state.current, self.dev

        def __exit__(self, *exc):
            state.current = self.before

    monkeypatch.setattr(sg, "_lib", Library(sg.lib(), state))
    monkeypatch.setattr(sg, "_on_gpu", lambda t, name: None)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state.current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev)
    return state


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def f32(*s):
    return torch.zeros(s)


def one():
    return sg.BlockWeight(u8(sg.packed_bytes(272, 144)), f32(2, 3), 272, 144)


def four():
    return sg.BlockWeight(u8(4 * sg.packed_bytes(272, 144)), f32(4, 2, 3), 272, 144, 4)


def plan():
    return sg.Routing(i32(5, 2), f32(5, 2), i32(5), i32(10), i32(5, 2))


CALLS = {
    "quant_act_block": lambda **s: sg.quant_act_block(bf(5, 272), **s),
    "quant_weight_block": lambda **s: sg.quant_weight_block(bf(4, 272, 144), **s),
    "pack_weight_block": lambda **s: sg.pack_weight_block(u8(272, 144), f32(3, 2), **s),
    "gemm_block": lambda **s: sg.gemm_block(u8(5, 272), f32(3, 5), one(), **s),
    "route_experts": lambda **s: sg.route_experts(f32(50, 8), 2, **s),
    "gemm_experts": lambda **s: sg.gemm_experts(u8(10, 272), f32(3, 10), four(), plan(), **s),
    "combine_experts": lambda **s: sg.combine_experts(bf(10, 144), plan(), **s),
}


@pytest.mark.parametrize("name", CALLS)
def test_gpu_and_stream(gpus, name):
    """A call runs with its tensors' GPU current, on that GPU's stream or a given one of it."""
    CALLS[name]()
    assert gpus.calls == [("ptpc_" + name, -1, 99)] and gpus.current == 0
    gpus.calls.clear()
    CALLS[name](stream=SimpleNamespace(device_index=-1, cuda_stream=7))
    assert gpus.calls == [("ptpc_" + name, -1, 7)]
    gpus.calls.clear()
    with pytest.raises(ValueError, match="stream: expected a stream of GPU -1"):
        CALLS[name](stream=SimpleNamespace(device_index=0, cuda_stream=7))
    assert not gpus.calls and gpus.current == 0
    gpus.status = 3
    with pytest.raises(sg.PtpcError) as e:
        CALLS[name]()
    assert e.value.status == 3 and "ptpc_" + name in str(e.value)


def raises(call, text, error=(ValueError, TypeError)):
    with pytest.raises(error, match=text):
        call()


def test_binding_quant(gpus):
    f = sg.quant_act_block
    raises(lambda: f(bf(5, 272).half()), "x: expected")
    raises(lambda: f(bf(5, 272, 1)), "x: expected a 2-D")
    raises(lambda: f(bf(272, 5).t()), "x: expected rows apart")
    raises(lambda: f(bf(1, 272).expand(5, 272)), "x: expected rows apart")
    raises(lambda: f(bf(5, 273), gate=True), "even number")
    raises(lambda: f(bf(5, 272), qx=u8(5, 256)), "qx: expected shape")
    raises(lambda: f(bf(5, 272), sx=f32(5, 3)), "sx: expected shape")
    raises(lambda: f(bf(5, 272), sx=f32(5, 3).t()), "sx: expected rows apart")
    raises(lambda: f(bf(5, 272), sx=torch.zeros(3, 5, dtype=torch.float64)), "sx: expected")
    raises(lambda: f(bf(5, 272), count=i32(2)), "count: expected")
    raises(lambda: f(bf(5, 272), count=i32(1).long()), "count: expected")
    assert not gpus.calls
    qx, sx = f(bf(5, 544), gate=True)
    assert qx.shape == (5, 272) and sx.shape == (3, 5)


def test_binding_weights(gpus):
    raises(lambda: sg.quant_weight_block(bf(272)), "w: expected")
    raises(lambda: sg.quant_weight_block(f32(272, 144)), "w: expected")
    raises(lambda: sg.quant_weight_block(bf(144, 272).t()), "w: expected rows apart")
    raises(lambda: sg.quant_weight_block(bf(1, 144).expand(272, 144)), "w: expected rows apart")
    f = sg.pack_weight_block
    raises(lambda: f(f32(272, 144), f32(3, 2)), "codes: expected")
    raises(lambda: f(u8(272), f32(3, 2)), "codes: expected")
    raises(lambda: f(u8(272, 144), f32(2, 3)), "scales: expected shape")
    raises(lambda: f(u8(272, 144), f32(3, 2).double()), "scales: expected")
    raises(lambda: f(u8(4, 272, 144), f32(3, 2)), "scales: expected shape")
    raises(lambda: f(u8(272, 288)[:, ::2], f32(3, 2)), "unit stride")
    assert not gpus.calls
    assert f(u8(144, 272).t(), f32(2, 3).t()).sw.shape == (2, 3)
    assert gpus.args[1:4] == (0, 1, 272)
    w = f(u8(4, 272, 144), f32(4, 3, 2))
    assert w.experts == 4 and w.sw.shape == (4, 2, 3) and w.data.numel() == 4 * 144 * 384
    n = sg.packed_bytes(272, 144)
    raises(lambda: sg.BlockWeight(u8(n - 1), f32(2, 3), 272, 144), "data: expected at least")
    raises(lambda: sg.BlockWeight(f32(n), f32(2, 3), 272, 144), "data: expected")
    raises(lambda: sg.BlockWeight(u8(n), f32(3, 2), 272, 144), "sw: expected")
    raises(lambda: sg.BlockWeight(u8(n), f32(4, 2, 3), 272, 144, 4), "data: expected at least")
    with pytest.raises(AttributeError, match="cannot be changed"):
        w.Ci = 16


def test_binding_products(gpus):
    f = sg.gemm_block
    q, s = u8(5, 272), f32(3, 5)
    raises(lambda: f(q, s, four()), "weight of one layer")
    raises(lambda: f(u8(5, 256), s, one()), "qx: expected shape")
    raises(lambda: f(q.float(), s, one()), "qx: expected")
    raises(lambda: f(q, f32(3, 4), one()), "sx: expected shape")
    raises(lambda: f(q, f32(2, 5), one()), "sx: expected shape")
    raises(lambda: f(q, s, one(), out=bf(4, 144)), "out: expected shape")
    raises(lambda: f(q, s, one(), out=f32(5, 144)), "out: expected")
    f = sg.gemm_experts
    q, s = u8(10, 272), f32(3, 10)
    raises(lambda: f(q, s, one(), plan()), "weight of experts")
    raises(lambda: f(u8(5, 272), f32(3, 5), four(), plan()), "qx: expected 10 rows")
    raises(lambda: f(q, s, four(), plan(), gather=True), "qx: expected 5 rows")
    raises(lambda: f(q, s, four(), sg.Routing(i32(5, 2), None, i32(4), i32(10), None)), "4 experts, got 3")
    raises(lambda: f(q, s, four(), sg.Routing(i32(5, 2), None, None, i32(10), None)), "offsets and rows")
    raises(lambda: f(q, s, four(), plan(), out=bf(5, 144)), "out: expected shape")
    assert not gpus.calls
    assert f(u8(5, 272), f32(3, 5), four(), plan(), gather=True).shape == (10, 144)
    assert gpus.args[8:12] == (2, 4, 5, 10)


def test_binding_routing(gpus):
    f = sg.route_experts
    x = f32(50, 8)
    raises(lambda: f(x.half(), 2), "logits: expected")
    raises(lambda: f(f32(8, 50).t(), 2), "logits: expected rows apart")
    raises(lambda: f(x, 2, scoring="relu"), "scoring: expected")
    raises(lambda: f(x, 2, bias=f32(7)), "bias: expected")
    raises(lambda: f(x, 2, bias=bf(8)), "bias: expected")
    raises(lambda: f(x, 0), "at least 1")
    raises(lambda: f(x, 2, first=8), "at least 1")
    raises(lambda: f(x, 2, workspace=u8(8)), "workspace: expected at least")
    assert not gpus.calls
    r = f(x, 2, first=2, local=3)
    assert r.ids.shape == r.slots.shape == r.weights.shape == (50, 2) and r.offsets.shape == (4,)
    assert r.rows.shape == (100,)
    raises(lambda: sg.Routing(None, None, i32(5), i32(10), None), "ids: expected")
    raises(lambda: sg.Routing(i32(10), None, None, None, None), "ids: expected")
    raises(lambda: sg.Routing(i32(5, 2), f32(5, 3), None, None, None), "weights: expected")
    raises(lambda: sg.Routing(i32(5, 2), None, i32(5, 1), None, None), "offsets: expected")
    raises(lambda: sg.Routing(i32(5, 2), None, i32(5), i32(9), None), "rows: expected")
    raises(lambda: sg.Routing(i32(5, 2).long(), None, None, None, None), "ids: expected")
    g = sg.combine_experts
    raises(lambda: g(bf(9, 144), plan()), "y: expected shape")
    raises(lambda: g(f32(10, 144), plan()), "y: expected")
    raises(lambda: g(bf(10, 144), plan(), out=bf(5, 128)), "out: expected shape")
    raises(lambda: g(bf(10, 144), sg.Routing(i32(5, 2), None, i32(5), i32(10), i32(5, 2))), "slots and weights")


def test_tensors_that_moved(gpus):
    """Storage exchanged behind a checked tensor, which no length was checked for."""
    q, s = u8(10, 272), f32(3, 10)
    for name in ("data", "sw"):
        bw, many = one(), four()
        getattr(bw, name).data = getattr(one(), name)[:0]
        getattr(many, name).data = getattr(four(), name)[:0]
        raises(lambda: sg.gemm_block(q, s, bw), "BlockWeight: its tensors lie elsewhere")
        raises(lambda: sg.gemm_experts(q, s, many, plan()), "BlockWeight: its tensors lie elsewhere")
    for name in ("offsets", "rows", "slots", "weights"):
        r = plan()
        getattr(r, name).data = getattr(plan(), name)[:0]
        raises(lambda: sg.gemm_experts(q, s, four(), r) if name in ("offsets", "rows")
               else sg.combine_experts(bf(10, 144), r), "Routing: its tensors lie elsewhere")
    assert not gpus.calls


def test_host_tensors_are_refused():
    for call in (lambda: sg.quant_act_block(bf(5, 272)), lambda: sg.quant_weight_block(bf(272, 144)),
                 lambda: sg.pack_weight_block(u8(272, 144), f32(3, 2)), lambda: one(), lambda: plan(),
                 lambda: sg.route_experts(f32(5, 8), 2)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()


# ---- the host layer under sanitizers ----------------------------------------------------

@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the ROCm headers not available")
def test_host_layer_under_sanitizers(tmp_path):
    exe = str(tmp_path / "block_fuzz")
    csrc = os.path.join(ROOT, "scaled_gemm_amd", "csrc")
    cmd = ["g++", "-std=c++20", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g",
           "-O1", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(ROOT, "tests", "sanitize", "block_fuzz.cpp"),
           os.path.join(csrc, "block_api.cpp"), os.path.join(csrc, "block_plan.cpp"), "-o", exe]
    for c in (cmd, [exe]):
        env = {k: v for k, v in os.environ.items() if k != "PTPC_FAULT"}
        r = subprocess.run(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, env=env)
        assert r.returncode == 0, r.stdout[-4000:]
    assert " 0 failures" in r.stdout, r.stdout
