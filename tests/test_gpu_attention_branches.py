"""Every branch of the attention calls' launch plans on the GPU: the 256-row prompt kernels, many
sequences, both joins of tiles, more ranges than a wave has lanes, one sequence in several
ranges, a workspace at its limit.  Inputs are large, so outputs are checked at sampled rows
against 64 bits (bounds: attention_ref.py), and whole where another kernel gives the same bits."""
import numpy as np
import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_gemm_amd
    scaled_gemm_amd.lib()
    return scaled_gemm_amd


def note(msg):
    print(msg, flush=True)


def normal(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32))


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def bounds(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


def sample(rng, n, most):
    """Up to `most` of n rows: the ends, the rows around tile edges, and others."""
    want = {0, n - 1, 31, 32, 63, 64} | {int(x) for x in rng.integers(0, max(n, 1), most)}
    rows = sorted(r for r in want if 0 <= r < n)
    return rows if len(rows) <= most else sorted(rng.choice(rows, most, replace=False).tolist())


# ---- prompts -----------------------------------------------------------------------------

def prompts(rng, T, Hq, Hk, D):
    x = normal(rng, T, (Hq + 2 * Hk) * D)
    x[:, :Hq * D] *= 2
    x = x.bfloat16()
    q, k, v = x.cuda().split([Hq * D, Hk * D, Hk * D], dim=1)
    return q.unflatten(1, (Hq, D)), k.unflatten(1, (Hk, D)), v.unflatten(1, (Hk, D))


def check_prompts(rng, got, q, k, v, lens, most):
    q, k, v, got = q.cpu(), k.cpu(), v.cpu(), got.cpu()
    for a, n in zip(bounds(lens), lens):
        rows = sample(rng, n, most)
        if rows:
            at = [a + r for r in rows]
            out, bound = ref.attend(q[at], k[a:a + n], v[a:a + n], [r + 1 for r in rows],
                                    ref.scale_of(q.shape[2]))
            ref.check(got[at], out, bound, f"prompt at {a} ({n} rows)")


@pytest.mark.parametrize("D", [64, 128])
def test_large_prompt_batch(sg, D):
    """T * q_heads above 2^18: the 256-row kernel.  A wave's 32 rows and the tiles of 64 keys are
    those of the 128-row kernel, which takes the same prompts one by one: the same bits."""
    Hq, Hk, lens = 128, 8, [700, 1, 900, 63, 0, 436]
    T = sum(lens)
    assert T * Hq >= 1 << 18 > max(lens) * Hq
    note(f"large prompt batch D={D}")
    rng = np.random.default_rng([D, 11])
    q, k, v = prompts(rng, T, Hq, Hk, D)
    got = sg.attn_prompt(q, k, v, i32(bounds(lens)))
    check_prompts(rng, got, q, k, v, lens, 8)
    for a, n in zip(bounds(lens), lens):
        if n:
            s = slice(a, a + n)
            one = sg.attn_prompt(q[s], k[s], v[s], i32([0, n]))
            assert torch.equal(one.view(torch.int16), got[s].view(torch.int16)), f"prompt at {a}"


@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("D", [64, 128])
def test_large_prompt_batch_with_a_bad_token(sg, D, what):
    """The 256-row kernel: a token that is not a number leaves earlier rows and other prompts
    as they were, bit for bit."""
    Hq, Hk, lens, at = 128, 8, [1100, 950, 300], 1100 + 612
    note(f"large prompt batch D={D} {what}")
    rng = np.random.default_rng([D, 12])
    q, k, v = (t.contiguous() for t in prompts(rng, sum(lens), Hq, Hk, D))
    cu = i32(bounds(lens))
    clean = sg.attn_prompt(q, k, v, cu).clone()
    v[at, 3] = float(what)
    k[at + 1, 3] = float("nan")
    got = sg.attn_prompt(q, k, v, cu)
    g = Hq // Hk
    heads = slice(3 * g, 4 * g)
    other = [h for h in range(Hq) if not 3 * g <= h < 4 * g]
    same = lambda a, b: torch.equal(a.contiguous().view(torch.int16),       # noqa: E731
                                    b.contiguous().view(torch.int16))
    assert same(got[:at], clean[:at]) and same(got[2050:], clean[2050:])
    assert same(got[:, other], clean[:, other])
    assert not torch.isfinite(got[at:2050, heads].float()).any()


def test_many_prompts(sg):
    """More prompts than a wave has lanes, empty ones among them."""
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(0, 40, 170)]
    lens[:3], lens[64:66], lens[-1] = [0, 0, 5], [0, 130], 0
    note("many prompts")
    q, k, v = prompts(rng, sum(lens), 6, 2, 64)
    got = sg.attn_prompt(q, k, v, i32(bounds(lens)))
    check_prompts(rng, got, q, k, v, lens, 6)


# ---- the paged cache -----------------------------------------------------------------------

def paged(sg, seed, nq, nkv, Hq, Hk, D, fp8, most, page=16, split=None, workspace=None):
    """Runs a paged call over a random cache and checks sampled rows of every sequence."""
    rng = np.random.default_rng(seed)
    pages, table = ref.paged_layout(rng, nkv, page)
    raw = []
    for _ in "kv":
        x = normal(rng, pages, Hk, page, D)
        raw.append(ref.quantize32(x.numpy()) if fp8 else (x.bfloat16(), None))
    (k, dk), (v, dv) = raw
    cache = sg.KVCache(*[None if t is None else t.cuda() for t in (k, v, dk, dv)])
    T = sum(nq)
    q = (2 * normal(rng, T, Hq, D)).bfloat16()
    need = sg.attn_paged_workspace_bytes(T, len(nq), max(nq), max(nkv), Hq, cache)
    if split is not None:
        assert (need > 0) == split, need
    if workspace is not None:
        assert workspace[0] <= need <= workspace[1], need
    got = sg.attn_paged(q.cuda(), i32(bounds(nq)), cache, table.cuda(), i32(nkv), max_q=max(nq),
                        max_kv=max(nkv),
                        out=torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16,
                                       device="cuda"))
    torch.cuda.synchronize()
    assert torch.isfinite(got.float()).all()
    got = got.cpu()
    for b, (a, n, m) in enumerate(zip(bounds(nq), nq, nkv)):
        rows = sample(rng, n, most)
        if not rows:
            continue
        j = np.arange(m)
        where = table[b].numpy()[j // page], slice(None), j % page
        val = [x[where[0], :, where[2]].double() if d is None else
               ref.e4m3_values(x[where[0], :, where[2]]) * d[where[0], :, where[2]].double()[..., None]
               for x, d in raw]
        at = [a + r for r in rows]
        out, bound = ref.attend(q[at], *val, [m - n + r + 1 for r in rows], ref.scale_of(D))
        ref.check(got[at], out, bound, f"sequence {b} ({n} rows, {m} keys)")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_many_chunks(sg, D, fp8):
    """More sequences than a wave has lanes in the tile kernel, some without new tokens."""
    rng = np.random.default_rng(14)
    nq = [int(x) for x in rng.integers(0, 13, 100)]
    nq[0], nq[7] = 0, 12
    nkv = [n + int(x) for n, x in zip(nq, rng.integers(0, 90, 100))]
    note(f"many chunks D={D} fp8={fp8}")
    paged(sg, [D, 14], nq, nkv, 8, 1, D, fp8, 12)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_parts_of_large_tiles(sg, fp8):
    """Tiles of 256 rows, split, more than 128 of them: joined 32 rows a workgroup."""
    note(f"many parts, 256 rows, fp8={fp8}")
    paged(sg, [15, fp8], [200, 150, 1, 250], [2600, 700, 2100, 250], 64, 8, 128, fp8, 5,
          split=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_parts_of_small_tiles(sg, fp8):
    """The same with tiles of 128 rows, more than 256 of them."""
    rng = np.random.default_rng(16)
    nq = [int(x) for x in rng.integers(1, 33, 32)]
    nq[3] = 32
    nkv = [n + int(x) for n, x in zip(nq, rng.integers(0, 400, 32))]
    nkv[5], nkv[20] = 3000, 1700
    note(f"many parts, 128 rows, fp8={fp8}")
    paged(sg, [16, fp8], nq, nkv, 32, 8, 64, fp8, 3, split=True)


@pytest.mark.parametrize("nq,nkv", [([1], [20000]), ([4], [30011]), ([1, 1], [17003, 9000])])
@pytest.mark.parametrize("fp8", [False, True])
def test_more_ranges_than_lanes(sg, nq, nkv, fp8):
    """A long context on one key head: 64 to 128 ranges of few rows, joined by one wave."""
    G, D = 8, 128
    note(f"many ranges nq={nq} nkv={nkv} fp8={fp8}")
    part = 4 * (D + 2) * G * max(nq)
    paged(sg, [sum(nkv), 17], nq, nkv, G, 1, D, fp8, 4, split=True,
          workspace=(65 * len(nq) * part, 128 * len(nq) * part))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [10, 20, 150])
def test_one_sequence_in_ranges(sg, n, D, fp8):
    """One sequence's chunk (80, 160 and 1200 rows a key head) over many keys: ranges by the
    plan for one sequence."""
    note(f"one sequence, {n} tokens, D={D} fp8={fp8}")
    paged(sg, [n, D, 18], [n], [5003], 8, 1, D, fp8, 7, page=32, split=True)


def test_workspace_at_its_limit(sg):
    """Ranges are made longer where their parts would take more than 2^28 bytes: 680 tiles would
    have three ranges each (2040 parts of 133120 bytes) and get two."""
    note("workspace limit")
    paged(sg, 19, [660, 640, 648, 644], [2000, 1400, 650, 900], 64, 8, 128, False, 4,
          split=True, workspace=(1360 * 133120, 1360 * 133120))
