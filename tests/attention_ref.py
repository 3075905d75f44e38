"""64-bit references of the attention operators, and the bounds their kernels
are held to (host side only, plain torch on the CPU).

Bound of an attention output, element by element.  With the weights p_j
(summing to 1), the exact output is o = sum p_j v_j; let A = sum p_j |v_j|.
  * the weights enter the MFMA as bf16: bf16 holds 8 significant bits, so a
    relative error of up to U = 2^-8 each (bf16_roundoff measures it), at most
    U A in all;
  * a score is an fp32 sum of D products: off by at most (D + 8) 2^-24 S
    with S = scale * sum |q_c k_c| (the 8: scaling, the key's scale, the
    change to powers of two and the exponential), which changes a weight by
    that factor, and the weights' sum again by as much;
  * sums over n keys in fp32: at most n 2^-24 A each for weights and outputs;
    a join of ranges or a rescale adds a few more roundings (counted as 64);
  * the output is rounded once to bf16: U |o|.
Each is a worst case, so their sum (times 1.01 for the products of the
small terms) holds for every element.
"""
import math

import numpy as np
import torch


U = 2.0 ** -8


def bf16_roundoff():
    """Largest relative error of rounding to bf16 over a binade: just below U."""
    x = 1.0 + torch.arange(1 << 16, dtype=torch.float64) * 2.0 ** -16
    return float(((x.to(torch.bfloat16).double() - x).abs() / x).max())


def e4m3_values(codes):
    """uint8 E4M3 codes -> float64 values."""
    return codes.view(torch.float8_e4m3fn).to(torch.float64)


def attend(q, k, v, visible, scale):
    """float64 attention of one sequence: q [n, Hq, D], k, v [m, Hk, D], visible [n] keys each
    row sees (the first ones).  Returns (out, bound) [n, Hq, D]."""
    n, Hq, D = q.shape
    m, Hk, _ = k.shape
    out = torch.zeros((n, Hq, D), dtype=torch.float64)
    bound = torch.zeros_like(out)
    q, k, v = q.double(), k.double(), v.double()
    for i in range(n):
        e = min(m, max(0, int(visible[i])))
        if e == 0:
            continue
        for h in range(Hq):
            hk = h * Hk // Hq
            kk, vv = k[:e, hk], v[:e, hk]
            s = scale * (kk @ q[i, h])
            S = abs(scale) * (kk.abs() @ q[i, h].abs()).max()
            p = torch.softmax(s, dim=0)
            out[i, h] = p @ vv
            A = p @ vv.abs()
            ds = (D + 8) * 2.0 ** -24 * float(S)
            rel = U + 2 * ds + (2 * e + 64) * 2.0 ** -24
            bound[i, h] = 1.01 * (rel * A + U * out[i, h].abs()) + 1e-38
    return out, bound


def check(got, out, bound, what):
    """A bf16 result against (out, bound)."""
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    bad = (got - out).abs() > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outputs outside the bound, "
                           f"worst {float(((got - out).abs() / bound.clamp_min(1e-300)).max()):.3g}x")
    zero = bound.amax(dim=-1) <= 1e-38
    assert (got[zero] == 0).all(), f"{what}: a row that sees nothing is not zero"


def rope_table(n, rot, base=10000.0):
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / max(rot, 1))
    a = np.arange(n, dtype=np.float64)[:, None] * f
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32))


def rotate32(x, table, pos, interleaved):
    """The rotation in fp32, every product and sum rounded by itself: numpy float32 [T, H, D]."""
    x = x.float().numpy().copy()
    r = table.shape[1]
    if r == 0:
        return x
    row = table.numpy()[pos.numpy()][:, None, :]
    c, s = row[..., :r // 2], row[..., r // 2:]
    ia = slice(0, r, 2) if interleaved else slice(0, r // 2)
    ib = slice(1, r, 2) if interleaved else slice(r // 2, r)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = b * c + a * s
    return x


def bits32_to_bf16(x):
    """float32 numpy -> torch.bfloat16, nearest even."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def quantize32(x):
    """The per-head rule on fp32 values [..., D]: (float8 codes as uint8 torch, scales)."""
    top = np.abs(x).max(axis=-1)
    dx = np.where(top == 0, np.float32(1), top / np.float32(448)).astype(np.float32)
    y = torch.from_numpy((x / dx[..., None]).astype(np.float32))
    return y.to(torch.float8_e4m3fn).view(torch.uint8), torch.from_numpy(dx)


def paged_layout(rng, kv_lens, page, extra=3, width=None):
    """A page table [B, width] over shuffled pages; entries past a sequence's pages are junk."""
    need = [-(-n // page) for n in kv_lens]
    pages = sum(need) + extra
    order = rng.permutation(pages).astype(np.int32)
    width = width or max(max(need), 1)
    table = np.full((len(kv_lens), width), -7, dtype=np.int32)
    a = 0
    for b, n in enumerate(need):
        table[b, :n] = order[a:a + n]
        a += n
    return pages, torch.from_numpy(table)


def scale_of(D):
    return 1.0 / math.sqrt(D)
