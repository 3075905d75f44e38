"""Every call of the binding runs with its tensors' GPU current, on a stream of that GPU (CPU
only: the library and torch's device calls are stand-ins, CPU tensors are those of GPU -1 and
GPU 0 is current)."""
from types import SimpleNamespace

import pytest
import torch

import scaled_gemm_amd as sg


class Library:
    """Size queries by the real library; every other call notes the current GPU and its stream."""

    def __init__(self, real, state):
        self.real, self.state = real, state

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*a):
            last = a[-1]
            self.state.calls.append((name, self.state.current,
                                     getattr(last, "value", last)))
            return self.state.status
        call.__name__ = name
        return call


@pytest.fixture
def gpus(monkeypatch):
    state = SimpleNamespace(current=0, calls=[], status=0)

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
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state.current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda dev=None: SimpleNamespace(
                            cuda_stream=100 + (state.current if dev is None else dev)))
    return state


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def weight(per_tensor=False):
    return sg.PackedWeight(u8(sg.packed_bytes(64, 48)), torch.zeros(1 if per_tensor else 48), 64,
                           48, per_tensor)


def cache():
    return sg.KVCache(bf(3, 2, 16, 64), bf(3, 2, 16, 64))


x, qx, dx, one = bf(6, 64), u8(6, 64), torch.zeros(6), torch.ones(1)
q, k = bf(5, 4, 64), bf(5, 2, 64)
CALLS = {
    "quant_act": lambda **s: sg.quant_act(x, **s),
    "quant_weight": lambda **s: sg.quant_weight(bf(64, 48), **s),
    "unpack_weight": lambda **s: sg.unpack_weight(weight(), **s),
    "gemm": lambda **s: sg.gemm(qx, dx, weight(), **s),
    "gemm_ws": lambda **s: sg.gemm_ws(qx, dx, weight(), **s),
    "gemm_noalloc": lambda **s: sg.gemm_noalloc(qx, dx, weight(), **s),
    "gemm_unfused": lambda **s: sg.gemm_unfused(qx, dx, weight(), **s),
    "gemm_unfused_bf16": lambda **s: sg.gemm_unfused_bf16(qx, dx, weight(), **s),
    "tensor_scale": lambda **s: sg.tensor_scale(x, **s),
    "quant_act_static": lambda **s: sg.quant_act_static(x, one, **s),
    "quant_weight_static": lambda **s: sg.quant_weight_static(bf(64, 48), one, **s),
    "gemm_tensor": lambda **s: sg.gemm_tensor(qx, one, weight(True), **s),
    "rope_append": lambda **s: sg.rope_append(q, k, k, torch.zeros(9, 64), i32(5), i32(5).long(),
                                              cache(), q_out=bf(5, 4, 64), **s),
    "attn_paged": lambda **s: sg.attn_paged(q, i32(3), cache(), i32(2, 6), i32(2),
                                            out=bf(5, 4, 64), **s),
    "attn_prompt": lambda **s: sg.attn_prompt(q, k, k, i32(3), out=bf(5, 4, 64), **s),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_gpu_is_current(gpus, name):
    CALLS[name]()
    assert gpus.calls == [("ptpc_" + name, -1, 99)]
    assert gpus.current == 0


@pytest.mark.parametrize("name", CALLS)
def test_a_given_stream(gpus, name):
    CALLS[name](stream=SimpleNamespace(device_index=-1, cuda_stream=7))
    assert gpus.calls == [("ptpc_" + name, -1, 7)]
    gpus.calls.clear()
    with pytest.raises(ValueError, match="stream: expected a stream of GPU -1"):
        CALLS[name](stream=SimpleNamespace(device_index=0, cuda_stream=7))
    assert not gpus.calls and gpus.current == 0


@pytest.mark.parametrize("name", CALLS)
def test_a_refused_call_raises(gpus, name):
    gpus.status = 3
    with pytest.raises(sg.PtpcError) as e:
        CALLS[name]()
    assert e.value.status == 3 and "ptpc_" + name in str(e.value) and gpus.current == 0


def test_the_current_gpu_is_left_alone(gpus, monkeypatch):
    """No switch where the tensors' GPU is current already."""
    gpus.current = -1
    monkeypatch.setattr(torch.cuda, "device", None)
    sg.quant_act(x)
    assert gpus.calls == [("ptpc_quant_act", -1, 99)]
