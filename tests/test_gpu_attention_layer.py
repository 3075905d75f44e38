"""The attention operators in the layer they are made for: prefill, decode steps and the same
tokens as one chunk, between the FP8 projections (examples/decoder_attention.py)."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


def example():
    spec = importlib.util.spec_from_file_location(
        "decoder_attention", os.path.join(ROOT, "examples", "decoder_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fp8_cache", [False, True])
@pytest.mark.parametrize("tokens,steps", [(300, 8), (17, 20)])
def test_steps_and_chunk_agree(tokens, steps, fp8_cache):
    """The two kernels' bf16 attention outputs differ by two roundings (the weights' and the
    output's, 2^-8 each) at most, in each; the O projection re-quantizes them to E4M3 (relative
    step 2^-3, half of it as error), so a difference may flip codes: the projected sums of 2048
    such terms, whose differences are independent, stay within 2^-4 of the largest output."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"layer tokens={tokens} steps={steps} fp8_cache={fp8_cache}", flush=True)
    assert example().run(tokens, steps, fp8_cache) <= 2.0 ** -4


def test_prompt_equals_paged_chunk():
    """A prompt through attn_prompt and through a bf16 cache: the same kernel on the same
    numbers, bit for bit."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_gemm_amd as sg
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    n, hq, hk, d, page = 777, 8, 2, 128, 16
    q, k, v = (torch.randn((n, h, d), device="cuda", generator=g).bfloat16() for h in (hq, hk, hk))
    cache = sg.kv_cache(50, hk, page, d)
    table = torch.randperm(50, device="cuda", generator=g).to(torch.int32)[None]
    at = torch.arange(n, device="cuda")
    slots = table[0, at // page].long() * page + at % page
    none = torch.zeros((1, 0), device="cuda")
    same = sg.rope_append(q, k, v, none, torch.zeros(n, dtype=torch.int32, device="cuda"), slots,
                          cache)
    assert torch.equal(same, q)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    a = sg.attn_prompt(q, k, v, cu)
    b = sg.attn_paged(q, cu, cache, table, cu[1:], max_q=n, max_kv=1)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
