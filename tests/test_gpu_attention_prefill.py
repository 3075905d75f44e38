"""The prefill of examples/decoder_attention.py: its attention against 64 bits, over the prompts
themselves and over what the cache holds of them, and the chunk of decoded tokens by the kernel
for many rows."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import attention_ref as ref
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location(
        "decoder_attention", os.path.join(ROOT, "examples", "decoder_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def cached(cache, table, m):
    """float64 keys and values of the first m tokens of a sequence."""
    j = torch.arange(m)
    p, off = table.cpu().long()[j // cache.page_size], j % cache.page_size
    out = []
    for x, d in ((cache.k, cache.dk), (cache.v, cache.dv)):
        x = x.cpu()[p, :, off]
        out.append(x.double() if d is None else
                   ref.e4m3_values(x) * d.cpu()[p, :, off].double()[..., None])
    return out


@pytest.mark.parametrize("fp8_cache", [False, True])
@pytest.mark.parametrize("lens", [[120, 40], [17, 5], [70, 64]])
def test_prefill(example, lens, fp8_cache):
    print(f"prefill lens={lens} fp8_cache={fp8_cache}", flush=True)
    import scaled_gemm_amd as sg
    ex = example
    layer = ex.AttentionLayer(len(lens), max(lens), fp8_cache)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    x = torch.randn((sum(lens), ex.HIDDEN), device="cuda", generator=g).bfloat16()
    got, q, cu = ex.prefill(layer, x, lens)
    paged = sg.attn_paged(q, cu, layer.cache, layer.table, ex.i32(lens), max_q=max(lens),
                          max_kv=max(lens))
    q0, k, v = (t.cpu() for t in layer.project(x))
    pos = torch.cat([torch.arange(m) for m in lens])
    turn = lambda t: ref.bits32_to_bf16(ref.rotate32(t, layer.rope.cpu(), pos, False))  # noqa: E731
    assert torch.equal(q.cpu().view(torch.int16), turn(q0).view(torch.int16))
    k, a = turn(k), 0
    for b, m in enumerate(lens):
        s = slice(a, a + m)
        see = np.arange(m) + 1
        out, bound = ref.attend(q[s].cpu(), k[s], v[s], see, ref.scale_of(ex.D))
        ref.check(got[s], out, bound, f"prompt {b}")
        out, bound = ref.attend(q[s].cpu(), *cached(layer.cache, layer.table[b], m), see,
                                ref.scale_of(ex.D))
        ref.check(paged[s], out, bound, f"prompt {b} from the cache")
        a += m


def test_prompt_and_bf16_cache_are_the_same_numbers(example):
    """The bf16 cache holds the rotated keys and the values as they are, and both calls run the
    kernel of many rows over the same tiles: no difference."""
    assert example.compare(300, 1, fp8_cache=False)[0] == 0.0


@pytest.mark.parametrize("fp8_cache", [False, True])
def test_steps_and_chunk_by_two_kernels(example, fp8_cache):
    """20 steps make 80 rows a key head: the chunk runs in the kernel of many rows, the steps in
    that of few.  Each rounds an output twice (weights and result, 2^-8 each); the O projection
    re-quantizes it (step 2^-3): the sums of 2048 terms stay within 2^-4 of the largest output."""
    assert example.run(300, 20, fp8_cache) <= 2.0 ** -4
