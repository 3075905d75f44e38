"""Corners of the attention operators on the GPU: tiny heads, scales of any sign, and values
that are not finite where some rows see them and others do not."""
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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [0, 3, 8, 12, 16])
def test_tiny_keys_stay_numbers(sg, D, power):
    """Keys near the smallest fp32 numbers: bf16 subnormals, rotated by a table whose cosines are
    2^-power.  amax / 448 then has few bits left, or none.  A cached value is within its E4M3
    step (2^-4 of it, or half the smallest step of 2^-9 scales) of the rotated one."""
    note(f"tiny keys D={D} power={power}")
    rng = np.random.default_rng([D, power])
    T, H = 12, 2
    bits = torch.from_numpy(rng.integers(1, 6, (T, H, D)).astype(np.int16))     # n * 2^-133
    k = bits.view(torch.bfloat16)
    k[3, 0] = 0
    v = bf16(rng, T, H, D)
    table = torch.zeros((1, D))
    table[:, :D // 2] = 2.0 ** -power
    cache = sg.kv_cache(1, H, 16, D, fp8=True)
    sg.rope_append(k[:, :0].cuda(), k.cuda(), v.cuda(), table.cuda(),
                   torch.zeros(T, dtype=torch.int32).cuda(), torch.arange(T).cuda(), cache)
    codes = ref.e4m3_values(cache.k.cpu())[0, :, :T].transpose(0, 1)
    scale = cache.dk.cpu().double()[0, :, :T].transpose(0, 1)[..., None]
    assert torch.isfinite(codes).all() and torch.isfinite(scale).all()
    want = k.double() * 2.0 ** -power
    want = (want / 2.0 ** -149).round() * 2.0 ** -149       # the rotation's fp32 product
    off = (codes * scale - want).abs()
    assert (off <= 1.01 * want.abs() * 2.0 ** -4 + scale * 2.0 ** -10).all()
    assert (scale[3, 0] == 1).all()


# ---- attention: one sequence among others, of any kernel -------------------------------

# (new tokens, cached tokens): with four query heads to a key head these are 12 rows (one tile of
# 16), 28 (one of 32), 48 (two tiles), 100 (a tile of 128 rows) and 280 (tiles of 256); the
# long ones have their keys split over workgroups.
SHAPES = {"few16": (3, 77), "few32": (7, 90), "few48": (12, 200), "tile128": (25, 130),
          "tile256": (70, 300), "few16 split": (3, 3000), "tile128 split": (25, 2600)}
G, HK = 4, 2


class Batch:
    """A cache with two sequences: the one that is looked at, and a short one beside it."""

    def __init__(self, sg, seed, n, m, D, fp8, page=16):
        rng = np.random.default_rng(seed)
        self.sg, self.D, self.fp8 = sg, D, fp8
        self.nq, self.nkv = [n, 2], [m, 40]
        pages, self.table = ref.paged_layout(rng, self.nkv, page)
        shape = (pages, HK, page, D)
        x = [rng.standard_normal(shape).astype(np.float32) for _ in "kv"]
        if fp8:
            (self.k, self.dk), (self.v, self.dv) = (ref.quantize32(t) for t in x)
        else:
            self.k, self.v = (torch.from_numpy(t).bfloat16() for t in x)
            self.dk = self.dv = None
        self.q = bf16(rng, n + 2, G * HK, D, gain=2.0)
        self.page = page

    def at(self, b, j):
        """Index of cached token j of sequence b."""
        return int(self.table[b, j // self.page]), slice(None), j % self.page

    def values(self, b, side):
        j = np.arange(self.nkv[b])
        rows = self.table[b].numpy()[j // self.page]
        x = getattr(self, side)[rows, :, j % self.page]
        if not self.fp8:
            return x.double()
        d = getattr(self, "d" + side)[rows, :, j % self.page]
        return ref.e4m3_values(x) * d.double()[..., None]

    def run(self, scale=None):
        up = lambda t: None if t is None else t.cuda()                       # noqa: E731
        cache = self.sg.KVCache(up(self.k), up(self.v), up(self.dk), up(self.dv))
        n = self.nq[0]
        if self.nkv[0] > 2000:
            assert self.sg.attn_paged_workspace_bytes(n + 2, 2, n, self.nkv[0], G * HK, cache) > 0
        got = self.sg.attn_paged(
            self.q.cuda(), torch.tensor([0, n, n + 2], dtype=torch.int32).cuda(), cache,
            self.table.cuda(), torch.tensor(self.nkv, dtype=torch.int32).cuda(),
            max_q=max(self.nq), max_kv=max(self.nkv), scale=scale,
            out=torch.full((n + 2, G * HK, self.D), 7.0, dtype=torch.bfloat16, device="cuda"))
        torch.cuda.synchronize()
        return got.cpu()

    def want(self, b, scale):
        n, m = self.nq[b], self.nkv[b]
        a = 0 if b == 0 else self.nq[0]
        return ref.attend(self.q[a:a + n], self.values(b, "k"), self.values(b, "v"),
                          [m - n + i + 1 for i in range(n)], scale)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.25])
def test_scales_of_any_sign(sg, shape, D, fp8, scale):
    n, m = SHAPES[shape]
    note(f"scale {scale} {shape} D={D} fp8={fp8}")
    b = Batch(sg, [n, m, D], n, m, D, fp8)
    got = b.run(scale)
    for s, rows in ((0, slice(0, n)), (1, slice(n, n + 2))):
        out, bound = b.want(s, scale)
        ref.check(got[rows], out, bound, f"sequence {s}")


@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.25])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_scales_of_any_sign(sg, D, scale):
    rng = np.random.default_rng([D, 5])
    n = 150
    q, k, v = bf16(rng, n, G * HK, D, gain=2.0), bf16(rng, n, HK, D), bf16(rng, n, HK, D)
    got = sg.attn_prompt(q.cuda(), k.cuda(), v.cuda(),
                         torch.tensor([0, n], dtype=torch.int32).cuda(), scale=scale)
    out, bound = ref.attend(q, k, v, np.arange(n) + 1, scale)
    ref.check(got, out, bound, "prompt")


def spoil(b, what, j):
    """Spoils cached token j of sequence 0 for key head 0 and returns the channels of an output row
    that sees it which cannot be finite (None: nothing can be said)."""
    p, _, off = b.at(0, j)
    every, some = slice(None), slice(8, 40, 3)
    if what.startswith("value"):
        if b.fp8:
            b.v[p, 0, off, some] = 0xFF if what == "value -inf" else 0x7F    # NaN either way
        else:
            b.v[p, 0, off, some] = float(what.split()[1])
        return some
    if what == "key nan":
        b.k[p, 0, off, 5] = 0x7F if b.fp8 else float("nan")
        return every
    if what == "key inf":
        if b.fp8:
            b.dk[p, 0, off] = float("inf")
        else:
            b.k[p, 0, off, 5] = float("inf")
        return None                     # minus infinity is a score like any other
    (b.dk if what == "key scale nan" else b.dv)[p, 0, off] = float(what.split()[-1])
    return every


WHAT = ["value nan", "value inf", "value -inf", "key nan", "key inf"]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("what,fp8", [(w, False) for w in WHAT] + [(w, True) for w in WHAT + [
    "key scale nan", "value scale nan", "value scale inf"]])
def test_what_only_some_rows_see(sg, shape, D, what, fp8):
    """One cached token of key head 0 is not a number: the middle new one, the last, or one that
    every row sees.  Rows that do not see it, other sequences and the other key head's rows are
    right to the bound; so are the channels of spoilt values' rows that hold numbers; the rest is
    not finite."""
    n, m = SHAPES[shape]
    note(f"nonfinite {what} {shape} D={D} fp8={fp8}")
    for j in (m - (n + 1) // 2, m - 1, m - n - 2):
        b = Batch(sg, [n, m, D, 3], n, m, D, fp8)
        clean = [b.want(s, ref.scale_of(D)) for s in (0, 1)]
        lost = spoil(b, what, j)
        got = b.run().double()
        ref.check(got[n:], *clean[1], f"the other sequence ({j})")
        got, (out, bound) = got[:n], clean[0]
        ref.check(got[:, G:], out[:, G:], bound[:, G:], f"the other key head ({j})")
        first = max(0, j - (m - n))     # the first row that sees token j
        ref.check(got[:first, :G], out[:first, :G], bound[:first, :G], f"rows before ({j})")
        if lost is None:
            continue
        sees = got[first:, :G]
        assert not torch.isfinite(sees[..., lost]).any(), f"rows that see it ({j})"
        keep = torch.ones(D, dtype=torch.bool)
        keep[lost] = False
        if keep.any():
            ref.check(sees[..., keep], out[first:, :G][..., keep], bound[first:, :G][..., keep],
                      f"channels beside it ({j})")
