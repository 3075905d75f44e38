"""The attention half of a decoder layer, prefill and decode, on PTPC-FP8 linear layers.

    python examples/decoder_attention.py [--tokens 300] [--steps 20] [--bf16-cache]

Two sequences of a small grouped-head layer (16 query heads on 4 key heads of 128):

  prefill   quantize the tokens, QKV projection, rotate and append to the paged cache,
            causal attention over the packed prompts, O projection;
  decode    the same for one new token per sequence, attention over the cache.

Both are computed a second way.  The prompts' attention is taken over the cache: the same
numbers if the cache is bf16, quantized keys and values if it is E4M3.  The decoded tokens are
recomputed as one chunk over the same cache, by another kernel from 17 steps on (more than 64
rows a key head; fewer run in the kernel of the single tokens).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scaled_gemm_amd as sg  # noqa: E402

HIDDEN, HQ, HK, D, PAGE = 2048, 16, 4, 128, 16


class AttentionLayer:
    """QKV and O projections with FP8 weights, a paged cache and its page table."""

    def __init__(self, sequences, max_tokens, fp8_cache, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(ci, co):
            w = torch.randn((ci, co), device="cuda", generator=g) * ci ** -0.5
            return sg.quant_weight(w.bfloat16())

        self.qkv, self.o = weight(HIDDEN, (HQ + 2 * HK) * D), weight(HQ * D, HIDDEN)
        per = -(-max_tokens // PAGE)
        self.cache = sg.kv_cache(sequences * per, HK, PAGE, D, fp8=fp8_cache)
        order = torch.randperm(sequences * per, device="cuda", generator=g)
        self.table = order.to(torch.int32).reshape(sequences, per)
        f = 500000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        a = torch.arange(max_tokens, device="cuda", dtype=torch.float64)[:, None] * f
        self.rope = torch.cat([a.cos(), a.sin()], dim=1).float()

    def project(self, x):
        """Hidden states [T, HIDDEN] -> q, k, v: slices of one FP8 projection's output."""
        y = sg.linear(x, self.qkv)
        q, k, v = y.split([HQ * D, HK * D, HK * D], dim=1)
        return q.unflatten(1, (HQ, D)), k.unflatten(1, (HK, D)), v.unflatten(1, (HK, D))

    def append(self, q, k, v, seq, pos):
        slots = self.table[seq, pos // PAGE].long() * PAGE + pos % PAGE
        return sg.rope_append(q, k, v, self.rope, pos.to(torch.int32), slots, self.cache)

    def output(self, a):
        return sg.linear(a.flatten(1), self.o)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prefill(layer, x, lens):
    """Attention of whole prompts, packed one after another in x [T, HIDDEN], their keys and
    values appended to the cache: (attention, rotated queries, bounds of the prompts)."""
    seq = torch.cat([torch.full((m,), b, device="cuda") for b, m in enumerate(lens)])
    pos = torch.cat([torch.arange(m, device="cuda") for m in lens])
    q, k, v = layer.project(x)
    q = layer.append(q, k, v, seq, pos)
    # Attention reads rotated keys, and the cache keeps the only copy (quantized, if it is E4M3):
    # the keys are rotated once more, as queries of a cache without pages.
    scratch = sg.kv_cache(0, HK, PAGE, D)
    kr = sg.rope_append(k, k, v, layer.rope, pos.to(torch.int32), torch.full_like(pos, -1), scratch)
    cu = i32([0] + [sum(lens[:b + 1]) for b in range(len(lens))])
    return sg.attn_prompt(q, kr, v, cu), q, cu


def difference(a, b):
    """Largest difference of two results, relative to the largest value."""
    return float((a.float() - b.float()).abs().max() / b.float().abs().max())


def compare(tokens=300, steps=20, fp8_cache=True, seed=1):
    """How far the two ways of the prefill's attention and of the decode steps' outputs differ."""
    lens = [tokens, max(1, tokens // 3)]
    n = len(lens)
    layer = AttentionLayer(n, tokens + steps, fp8_cache)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    draw = lambda t: torch.randn((t, HIDDEN), device="cuda", generator=g).bfloat16()  # noqa: E731

    prompt, q, cu = prefill(layer, draw(sum(lens)), lens)
    assert torch.isfinite(layer.output(prompt).float()).all()
    cached = sg.attn_paged(q, cu, layer.cache, layer.table, i32(lens), max_q=tokens,
                           max_kv=tokens)

    # decode: one token per sequence and step
    one = i32(list(range(n + 1)))
    every = torch.arange(n, device="cuda")
    outs, queries = [], []
    for s in range(steps):
        q, k, v = layer.project(draw(n))
        at = torch.tensor([m + s for m in lens], device="cuda")
        q = layer.append(q, k, v, every, at)
        a = sg.attn_paged(q, one, layer.cache, layer.table, (at + 1).to(torch.int32), max_q=1,
                          max_kv=max(lens) + s + 1)
        outs.append(layer.output(a))
        queries.append(q)

    # the same tokens as one chunk of each sequence
    q = torch.stack(queries, dim=1).flatten(0, 1)
    a = sg.attn_paged(q, i32([b * steps for b in range(n + 1)]), layer.cache, layer.table,
                      i32([m + steps for m in lens]), max_q=steps, max_kv=max(lens) + steps)
    chunk = layer.output(a).unflatten(0, (n, steps))
    stepwise = torch.stack(outs, dim=1)
    assert torch.isfinite(stepwise.float()).all()
    return difference(cached, prompt), difference(chunk, stepwise)


def run(tokens=300, steps=20, fp8_cache=True, seed=1):
    """How far decode steps and chunk differ, relative to the largest output."""
    return compare(tokens, steps, fp8_cache, seed)[1]


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=300)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--bf16-cache", action="store_true")
    a = p.parse_args()
    prompt, decode = compare(a.tokens, a.steps, fp8_cache=not a.bf16_cache)
    print(f"prefill of {a.tokens} + {max(1, a.tokens // 3)} tokens: prompt and cache differ by "
          f"{prompt:.2e} of the largest value; {a.steps} decode steps: steps and chunk by "
          f"{decode:.2e}", flush=True)


if __name__ == "__main__":
    main()
