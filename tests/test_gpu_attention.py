"""The attention operators on the GPU against 64-bit references.

Rotation and appending are bit-exact (fp32 products and sums rounded by
themselves, one rounding to bf16, the library's E4M3 rule); attention outputs
lie within the bound derived in attention_ref.py, element by element.
"""
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


def bf16(rng, *shape, gain=1.0):
    return torch.from_numpy((gain * rng.standard_normal(shape)).astype(np.float32)).bfloat16()


# ---- rotation and appending --------------------------------------------------------

@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter,page,fp8", [
    (1, 1, 1, 64, 64, False, 16, False),
    (1, 32, 8, 128, 128, False, 16, True),
    (33, 8, 2, 128, 64, True, 32, False),
    (70, 3, 3, 64, 16, False, 16, True),
    (257, 28, 4, 128, 128, True, 64, True),
    (19, 0, 2, 64, 0, False, 16, False),
    (130, 5, 1, 128, 48, False, 128, False),
])
def test_rope_append(sg, T, Hq, Hk, D, rot, inter, page, fp8):
    note(f"rope_append T={T} Hq={Hq} Hk={Hk} D={D} rot={rot} inter={inter} page={page} fp8={fp8}")
    rng = np.random.default_rng([T, Hq, Hk, D, rot])
    # slices of one wider row, the pitch not a multiple of the heads
    W = (Hq + 2 * Hk) * D + 24
    x = bf16(rng, T, W, gain=3.0)
    x[T // 2, Hq * D:Hq * D + D] = 0                      # an all-zero key head
    q = x[:, :Hq * D].unflatten(1, (Hq, D)) if Hq else torch.empty((T, 0, D), dtype=torch.bfloat16)
    k = x[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    v = x[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].unflatten(1, (Hk, D))
    table = ref.rope_table(400, rot)
    pos = torch.from_numpy(rng.integers(0, 400, T).astype(np.int32))
    pages = -(-T // page) + 2
    slots = torch.from_numpy(rng.permutation(pages * page)[:T].astype(np.int64))
    slots[0::7] = -1 if T > 1 else slots[0::7]
    if T > 3:
        slots[3] = pages * page                            # past the cache
        slots[2] = 1 << 40
    shape = (pages, Hk, page, D)
    if fp8:
        kc, vc = (torch.from_numpy(rng.integers(0, 120, shape).astype(np.uint8)) for _ in "kv")
        dk, dv = (torch.from_numpy(rng.random(shape[:3]).astype(np.float32)) for _ in "kv")
    else:
        kc, vc, dk, dv = bf16(rng, *shape), bf16(rng, *shape), None, None
    up = lambda t: t.cuda() if t is not None else None     # noqa: E731
    cache = sg.KVCache(up(kc), up(vc), up(dk), up(dv))
    xd = x.cuda()
    qd = xd[:, :Hq * D].unflatten(1, (Hq, D)) if Hq else q.cuda()
    kd = xd[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    vd = xd[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].unflatten(1, (Hk, D))
    got = sg.rope_append(qd, kd, vd, table.cuda(), pos.cuda(), slots.cuda(), cache,
                         interleaved=inter)
    torch.cuda.synchronize()
    want_q = ref.bits32_to_bf16(ref.rotate32(q, table, pos, inter))
    assert torch.equal(got.cpu().view(torch.int16), want_q.view(torch.int16)), "queries"
    for name, new, data, scale, dev, devs in (
            ("keys", ref.rotate32(k, table, pos, inter), kc, dk, cache.k, cache.dk),
            ("values", v.float().numpy(), vc, dv, cache.v, cache.dv)):
        want, wants = data.clone(), scale.clone() if fp8 else None
        codes, dx = ref.quantize32(new) if fp8 else (ref.bits32_to_bf16(new), None)
        for t in range(T):
            s = int(slots[t])
            if 0 <= s < pages * page:
                want[s // page, :, s % page] = codes[t]
                if fp8:
                    wants[s // page, :, s % page] = dx[t]
        eq = (torch.equal(dev.cpu(), want) if fp8 else
              torch.equal(dev.cpu().view(torch.int16), want.view(torch.int16)))
        assert eq, name
        if fp8:
            assert torch.equal(devs.cpu(), wants), name + " scales"


def test_rope_append_in_place_and_unknown_position(sg):
    rng = np.random.default_rng(5)
    T, H, D = 9, 2, 128
    q, k, v = bf16(rng, T, H, D), bf16(rng, T, H, D), bf16(rng, T, H, D)
    table = ref.rope_table(16, D)
    pos = torch.arange(T, dtype=torch.int32)
    cache = sg.kv_cache(2, H, 16, D)
    cache.k.zero_(), cache.v.zero_()
    qd, p2 = q.cuda(), pos.clone()
    p2[4], p2[6] = 16, -1
    out = sg.rope_append(qd, k.cuda(), v.cuda(), table.cuda(), p2.cuda(),
                         torch.arange(T).cuda(), cache, q_out=qd)
    assert out.data_ptr() == qd.data_ptr()
    known = [t for t in range(T) if t not in (4, 6)]
    want = ref.bits32_to_bf16(ref.rotate32(q, table, pos, False))
    assert torch.equal(qd.cpu()[known], want[known])
    assert torch.isnan(qd.cpu()[[4, 6]].float()).all()
    assert torch.isnan(cache.k[0, :, 4].float()).all() and not torch.isnan(cache.v.float()).any()


# ---- attention -----------------------------------------------------------------------

def make_cache(sg, rng, pages, Hk, page, D, fp8):
    """A full cache and its float64 values (k, v) [pages, Hk, page, D]."""
    shape = (pages, Hk, page, D)
    if not fp8:
        k, v = bf16(rng, *shape), bf16(rng, *shape)
        return sg.KVCache(k.cuda(), v.cuda()), k.double(), v.double()
    out, vals = [], []
    for _ in range(2):
        codes, dx = ref.quantize32(rng.standard_normal(shape).astype(np.float32))
        out.append((codes, dx))
        vals.append(ref.e4m3_values(codes) * dx.double()[..., None])
    (k, dk), (v, dv) = out
    return sg.KVCache(k.cuda(), v.cuda(), dk.cuda(), dv.cuda()), vals[0], vals[1]


def run_paged(sg, seed, nq, nkv, Hq, Hk, D, page, fp8, max_q=None, max_kv=None, gain=2.0,
              spoil=True, pad=0, width=None):
    rng = np.random.default_rng(seed)
    pages, table = ref.paged_layout(rng, nkv, page, width=width)
    cache, kval, vval = make_cache(sg, rng, pages, Hk, page, D, fp8)
    if spoil:       # everything no sequence owns holds NaN
        own = torch.zeros((pages, page), dtype=torch.bool)
        for b, m in enumerate(nkv):
            for j in range(m):
                own[table[b, j // page], j % page] = True
        spoilt = ~own[:, None, :].expand(pages, Hk, page).cuda()
        for t in (cache.k, cache.v):
            t[spoilt] = 0x7F if fp8 else float("nan")
        if fp8:
            cache.dk[spoilt] = float("inf")
            cache.dv[spoilt] = float("nan")
    T = sum(nq)
    cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    q = bf16(rng, T, Hq * D + pad, gain=gain)
    qd = q.cuda()[:, :Hq * D].unflatten(1, (Hq, D))
    q = q[:, :Hq * D].unflatten(1, (Hq, D))
    got = sg.attn_paged(qd, torch.from_numpy(cu).cuda(), cache, table.cuda(),
                        torch.tensor(nkv, dtype=torch.int32).cuda(),
                        max_q=max(nq) if max_q is None else max_q,
                        max_kv=max(nkv) if max_kv is None else max_kv,
                        out=torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16,
                                       device="cuda"))
    torch.cuda.synchronize()
    for b, (n, m) in enumerate(zip(nq, nkv)):
        j = np.arange(m)
        rows = table[b].numpy()[j // page], j % page
        k = kval[rows[0], :, rows[1]]
        v = vval[rows[0], :, rows[1]]
        vis = [m - n + i + 1 for i in range(n)]
        a = int(cu[b])
        out, bound = ref.attend(q[a:a + n], k, v, vis, ref.scale_of(D))
        ref.check(got[a:a + n], out, bound, f"sequence {b} ({n} rows, {m} keys)")
    return got


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 2, 128), (4, 4, 64), (7, 1, 128), (16, 1, 64),
                                     (20, 1, 128)])
@pytest.mark.parametrize("page", [16, 128])
def test_paged_single_tokens(sg, Hq, Hk, D, page, fp8):
    nkv = [1, 0, 15, 16, 17, 33, 64, 127, 300, 1000, 5]
    note(f"paged decode Hq={Hq} Hk={Hk} D={D} page={page} fp8={fp8}")
    run_paged(sg, [Hq, D, page, fp8], [1] * len(nkv), nkv, Hq, Hk, D, page, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hk,D,page", [(8, 2, 128, 16), (6, 2, 64, 32), (7, 1, 128, 64)])
def test_paged_few_tokens(sg, Hq, Hk, D, page, fp8):
    """2 .. 9 new tokens, ragged; one sequence shorter than its new tokens (rows that see
    nothing), one with exactly them."""
    nq = [5, 2, 9, 1, 7, 3]
    nkv = [77, 2, 4, 200, 7, 511]
    note(f"paged few Hq={Hq} Hk={Hk} D={D} page={page} fp8={fp8}")
    run_paged(sg, [Hq, D, page, 3], nq, nkv, Hq, Hk, D, page, fp8, pad=8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hk,D,page", [(4, 1, 128, 16), (2, 2, 64, 32), (3, 1, 128, 64)])
def test_paged_chunks(sg, Hq, Hk, D, page, fp8):
    """Chunks of a prompt: tiles that end inside, lengths around tile edges, no new tokens."""
    nq = [130, 0, 64, 33, 257, 100]
    nkv = [130, 40, 300, 800, 259, 90]
    note(f"paged chunks Hq={Hq} Hk={Hk} D={D} page={page} fp8={fp8}")
    run_paged(sg, [Hq, D, page, 4], nq, nkv, Hq, Hk, D, page, fp8, pad=16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nq,nkv", [([1], [4099]), ([1, 1, 1], [6000, 3, 2500]), ([6], [5000]),
                                    ([40, 2], [4500, 4100])])
def test_paged_long_context(sg, nq, nkv, fp8):
    """Few rows over many keys: the keys are split over workgroups and joined."""
    note(f"paged long nq={nq} nkv={nkv} fp8={fp8}")
    run_paged(sg, [sum(nkv), 9], nq, nkv, 4, 1, 128, 16, fp8)


@pytest.mark.parametrize("max_q,max_kv", [(1, 1), (1, 100000), (500, 1), (2, 64)])
def test_paged_bounds_need_not_be_tight(sg, max_q, max_kv):
    """max_q and max_kv size the launch, not the result."""
    note(f"paged hints max_q={max_q} max_kv={max_kv}")
    run_paged(sg, 12, [3, 40, 1], [700, 1500, 33], 8, 2, 128, 16, False, max_q=max_q,
              max_kv=max_kv)


def test_paged_peaked_and_flat_scores(sg):
    """Scores so far apart that all but one weight underflow, and all-equal scores."""
    run_paged(sg, 21, [1, 4, 70], [513, 600, 640], 4, 2, 128, 32, False, gain=60.0)
    run_paged(sg, 22, [1, 4, 70], [513, 600, 640], 4, 2, 128, 32, True, gain=0.0)


def test_paged_pages_outside_the_cache_stay_inside(sg):
    """Junk page numbers and lengths are cut to the buffers (the result is not defined)."""
    rng = np.random.default_rng(3)
    cache, _, _ = make_cache(sg, rng, 4, 2, 16, 128, False)
    table = torch.tensor([[0, 1 << 30], [-5, 2]], dtype=torch.int32).cuda()
    q = bf16(rng, 3, 4, 128).cuda()
    cu = torch.tensor([0, 1, 3], dtype=torch.int32).cuda()
    out = sg.attn_paged(q, cu, cache, table, torch.tensor([500, 31], dtype=torch.int32).cuda(),
                        max_q=2, max_kv=32)
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("Hq,Hk,D", [(4, 1, 128), (3, 3, 64), (14, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("lens", [[1], [77], [64, 1, 63, 0, 65, 130], [300, 17, 129], [1] * 40,
                                  [520]])
def test_prompt(sg, Hq, Hk, D, lens):
    note(f"prompt Hq={Hq} Hk={Hk} D={D} lens={lens[:8]}")
    rng = np.random.default_rng([Hq, D, sum(lens)])
    T = sum(lens)
    W = (Hq + 2 * Hk) * D + 8
    x = bf16(rng, T, W)
    x[:, :Hq * D] *= 2
    cut = lambda t: (t[:, :Hq * D].unflatten(1, (Hq, D)),                     # noqa: E731
                     t[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)),
                     t[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].unflatten(1, (Hk, D)))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    got = sg.attn_prompt(*cut(x.cuda()), torch.from_numpy(cu).cuda(),
                         out=torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16,
                                        device="cuda"))
    torch.cuda.synchronize()
    q, k, v = cut(x)
    for b, n in enumerate(lens):
        a = int(cu[b])
        out, bound = ref.attend(q[a:a + n], k[a:a + n], v[a:a + n], np.arange(n) + 1,
                                ref.scale_of(D))
        ref.check(got[a:a + n], out, bound, f"prompt {b} ({n} rows)")


@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
def test_later_tokens_never_reach_earlier_rows(sg, what):
    """NaN and infinities in the keys and values of later tokens leave earlier rows alone."""
    rng = np.random.default_rng(8)
    n, Hq, Hk, D, at = 150, 4, 2, 128, 90
    q, k, v = bf16(rng, n, Hq, D), bf16(rng, n, Hk, D), bf16(rng, n, Hk, D)
    out, bound = ref.attend(q[:at], k[:at], v[:at], np.arange(at) + 1, ref.scale_of(D))
    k[at, 0], v[at:at + 2] = float(what), float(what)
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    got = sg.attn_prompt(q.cuda(), k.cuda(), v.cuda(), cu)
    ref.check(got[:at], out, bound, "rows before")
    assert not torch.isfinite(got[at:].float()).any(dim=-1).any(), "rows that see them"
    page = 16
    pages, table = ref.paged_layout(rng, [n], page)
    cache = sg.kv_cache(pages, Hk, page, D)
    j = torch.arange(n)
    for dst, src in ((cache.k, k), (cache.v, v)):
        dst.zero_()
        dst[table[0, j // page].long().cuda(), :, (j % page).cuda()] = src.cuda()
    for n_new in (n, 62):      # all rows, and a tail whose first rows end before the token
        got = sg.attn_paged(q[n - n_new:].cuda(),
                            torch.tensor([0, n_new], dtype=torch.int32).cuda(), cache,
                            table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                            max_q=n_new)
        lo = n - n_new
        ref.check(got[:at - lo], out[lo:], bound[lo:], f"paged rows before ({n_new} new)")
        assert not torch.isfinite(got[at - lo:].float()).any(dim=-1).any()


def test_empty_calls(sg):
    z = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")       # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")       # noqa: E731
    assert sg.attn_prompt(z(0, 4, 64), z(0, 2, 64), z(0, 2, 64), i32(0)).shape == (0, 4, 64)
    cache = sg.kv_cache(1, 2, 16, 64)
    out = sg.attn_paged(z(0, 4, 64), i32(0), cache,
                        torch.empty((0, 1), dtype=torch.int32, device="cuda"), i32())
    assert out.shape == (0, 4, 64)
    sg.rope_append(z(0, 4, 64), z(0, 2, 64), z(0, 2, 64), torch.zeros((4, 64)).cuda(), i32(),
                   torch.empty(0, dtype=torch.int64, device="cuda"), cache)
    # a cache without pages, a table without columns: rows that see nothing
    none = sg.kv_cache(0, 2, 16, 64)
    out = sg.attn_paged(torch.ones((2, 4, 64), dtype=torch.bfloat16, device="cuda"), i32(0, 1, 2),
                        none, torch.empty((2, 0), dtype=torch.int32, device="cuda"), i32(0, 3))
    assert (out == 0).all()


def test_another_stream_and_workspace(sg):
    """The call runs on the stream it is given, with a caller's workspace, over a table whose
    rows are slices of a wider one."""
    rng = np.random.default_rng(31)
    cache, kval, vval = make_cache(sg, rng, 40, 1, 16, 128, False)
    wide = torch.from_numpy(rng.permutation(40).astype(np.int32)).reshape(1, 40).cuda()
    q = bf16(rng, 1, 4, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n = 600
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32).cuda()
    need = sg.attn_paged_workspace_bytes(1, 1, 1, n, 4, cache)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    qd = q.cuda()
    torch.cuda.synchronize()
    a = sg.attn_paged(qd, cu, cache, wide[:, :38], lens, max_q=1, max_kv=n, workspace=ws, stream=s)
    s.synchronize()
    b = sg.attn_paged(qd, cu, cache, wide[:, :38], lens, max_q=1, max_kv=n)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    assert (ws[need:] == 0xFF).all(), "written past the workspace"
    j = torch.arange(n)
    p = wide[0].cpu()[j // 16].long()
    out, bound = ref.attend(q, kval[p, :, j % 16], vval[p, :, j % 16], [n], ref.scale_of(128))
    ref.check(a, out, bound, "other stream")


def test_one_token_of_an_odd_row(sg):
    """A single token's pitch says nothing: a slice of a row whose width is no multiple of 8."""
    rng = np.random.default_rng(61)
    wide = torch.zeros((4, 3 * 64 + 5), dtype=torch.bfloat16)
    x = bf16(rng, 1, 3, 64)
    wide[:1, :192] = x.flatten(1)
    cut = torch.as_strided(wide.cuda(), (1, 3, 64), (197, 64, 1))
    assert cut.stride(0) % 8 != 0
    cu = torch.tensor([0, 1], dtype=torch.int32).cuda()
    got = sg.attn_prompt(cut[:, :1], cut[:, 1:2], cut[:, 2:], cu)
    assert torch.equal(got.cpu(), x[:, 2:])
    cache = sg.kv_cache(1, 1, 16, 64)
    q = sg.rope_append(cut[:, :1], cut[:, 1:2], cut[:, 2:], torch.zeros((1, 0)).cuda(),
                       torch.zeros(1, dtype=torch.int32).cuda(),
                       torch.zeros(1, dtype=torch.int64).cuda(), cache)
    assert torch.equal(q.cpu(), x[:, :1])
    got = sg.attn_paged(cut[:, :1], cu, cache, torch.zeros((1, 1), dtype=torch.int32).cuda(),
                        torch.ones(1, dtype=torch.int32).cuda())
    assert torch.equal(got.cpu(), x[:, 2:])


def test_long_cache_offsets(sg):
    """Pages whose bytes lie past 2^32 and 2^33 of the cache."""
    pages, Hk, page, D = 66000, 4, 128, 128           # 8.65 GB a side
    rng = np.random.default_rng(77)
    k, v = (torch.empty((pages, Hk, page, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    ids = [65999, 32769, 16385, 1]
    vals = [bf16(rng, len(ids), Hk, page, D) for _ in "kv"]
    for t, x in zip((k, v), vals):
        t[torch.tensor(ids).cuda()] = x.cuda()
    cache = sg.KVCache(k, v)
    n = 4 * page - 5
    for nq in (1, 80):
        q = bf16(rng, nq, 4, D)
        got = sg.attn_paged(q.cuda(), torch.tensor([0, nq], dtype=torch.int32).cuda(), cache,
                            torch.tensor([ids], dtype=torch.int32).cuda(),
                            torch.tensor([n], dtype=torch.int32).cuda(), max_q=nq)
        kk, vv = (x.transpose(1, 2).reshape(-1, Hk, D)[:n] for x in vals)
        out, bound = ref.attend(q, kk, vv, [n - nq + i + 1 for i in range(nq)], ref.scale_of(D))
        ref.check(got, out, bound, f"far pages, {nq} rows")
    x = bf16(rng, 2, 3 * Hk, D)
    slots = torch.tensor([65998 * page + 7, 40000 * page + 1]).cuda()
    sg.rope_append(x[:, :Hk].cuda(), x[:, Hk:2 * Hk].cuda(), x[:, 2 * Hk:].cuda(),
                   torch.zeros((1, 0)).cuda(), torch.zeros(2, dtype=torch.int32).cuda(), slots,
                   cache)
    assert torch.equal(k[65998, :, 7].cpu(), x[0, Hk:2 * Hk])
    assert torch.equal(v[40000, :, 1].cpu(), x[1, 2 * Hk:])


def test_graph_replay(sg):
    """Append and attention captured in one graph; replays follow their inputs' values."""
    rng = np.random.default_rng(41)
    B, Hq, Hk, D, page = 3, 8, 2, 128, 16
    cache, _, _ = make_cache(sg, rng, 64, Hk, page, D, True)
    table = torch.from_numpy(rng.permutation(63).astype(np.int32).reshape(B, 21)).cuda()
    rope = ref.rope_table(400, D).cuda()
    x = bf16(rng, B, Hq + 2 * Hk, D).cuda()
    pos = torch.tensor([5, 100, 330], dtype=torch.int32).cuda()
    slots = torch.zeros(B, dtype=torch.int64).cuda()
    lens = torch.zeros(B, dtype=torch.int32).cuda()
    cu = torch.arange(B + 1, dtype=torch.int32).cuda()
    qr = torch.empty((B, Hq, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(1, sg.attn_paged_workspace_bytes(B, B, 1, 21 * page, Hq, cache)),
                     dtype=torch.uint8, device="cuda")

    def step():
        sg.rope_append(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], rope, pos, slots, cache,
                       q_out=qr)
        sg.attn_paged(qr, cu, cache, table, lens, max_q=1, out=out, workspace=ws)

    def advance(i):
        x.copy_(bf16(np.random.default_rng([41, i]), B, Hq + 2 * Hk, D))
        pos.add_(1)
        p = pos.long()
        slots.copy_(table.long()[torch.arange(B).cuda(), p // page] * page + p % page)
        lens.copy_(pos + 1)

    advance(0)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        step()
    for i in range(1, 5):
        advance(i)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        a = out.clone()
        kc = cache.k.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(kc, cache.k), f"replay {i}"
        torch.randn(1 << 20, device="cuda").sum().item()
