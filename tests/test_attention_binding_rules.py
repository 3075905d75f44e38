"""Rules of the attention binding beyond its shape checks (CPU only; the library's calls are
stand-ins that note their arguments)."""
import pytest
import torch

import scaled_gemm_amd as sg


class Library:
    """Size queries by the real library; every other call is noted and succeeds."""

    def __init__(self, real, calls):
        self.real, self.calls = real, calls

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*a):
            self.calls.append((name, a))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    noted = []
    monkeypatch.setattr(sg, "_lib", Library(sg.lib(), noted))
    monkeypatch.setattr(sg, "_on_gpu", lambda t, name: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    return noted


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def cache():
    return sg.KVCache(bf(3, 2, 16, 64), bf(3, 2, 16, 64))


def test_rows_of_no_sequence_are_refused(calls):
    """Without a sequence nothing would write the rows' outputs."""
    with pytest.raises(ValueError, match="no sequence"):
        sg.attn_prompt(bf(5, 4, 64), bf(5, 2, 64), bf(5, 2, 64), i32(1))
    with pytest.raises(ValueError, match="no sequence"):
        sg.attn_paged(bf(5, 4, 64), i32(1), cache(), i32(0, 6), i32(0))
    assert not calls
    assert sg.attn_prompt(bf(0, 4, 64), bf(0, 2, 64), bf(0, 2, 64), i32(1)).shape == (0, 4, 64)
    assert sg.attn_paged(bf(0, 4, 64), i32(1), cache(), i32(0, 6), i32(0)).shape == (0, 4, 64)
