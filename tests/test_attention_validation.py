"""Refusals of the attention operators (CPU only): the C ABI before any HIP
call, and the Python binding before any call of the library."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import scaled_gemm_amd as sg
from conftest import ROOT

OK, NULLP, SHAPE, UNSUPPORTED, ALIGN, HIP = range(6)
A, B, C, D, E, F, G = (0x10000 * i for i in range(1, 8))      # never dereferenced
MIS = 0x10008


def cache(k=A, v=B, dk=None, dv=None, pages=4, heads=2, page=16, d=128, fp8=0):
    return sg._CacheStruct(k, v, dk, dv, pages, heads, page, d, fp8)


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    """Whatever passes validation reports PTPC_ERR_HIP instead of launching."""
    monkeypatch.setenv("PTPC_FAULT", "launch")


def append(c=None, **kw):
    a = dict(q=C, ldq=512, k=D, ldk=256, v=E, ldv=256, table=F, n_pos=100, rot=128, inter=0,
             pos=G, slots=G, T=3, hq=4, out=C, ldqo=512)
    a.update(kw)
    return sg.lib().ptpc_rope_append(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"],
                                     a["table"], a["n_pos"], a["rot"], a["inter"], a["pos"],
                                     a["slots"], a["T"], a["hq"], c or cache(), a["out"],
                                     a["ldqo"], None)


def paged(c=None, **kw):
    a = dict(q=C, ldq=512, cu=D, table=E, ldt=8, width=8, lens=F, T=3, B=3, max_q=1, max_kv=100,
             hq=4, out=G, ldo=512, ws=A, nb=1 << 40)
    a.update(kw)
    return sg.lib().ptpc_attn_paged(a["q"], a["ldq"], a["cu"], c or cache(), a["table"], a["ldt"],
                                    a["width"], a["lens"], a["T"], a["B"], a["max_q"],
                                    a["max_kv"], a["hq"], 0.1, a["out"], a["ldo"], a["ws"],
                                    a["nb"], None)


def prompt(**kw):
    a = dict(q=A, ldq=512, k=B, ldk=256, v=C, ldv=256, cu=D, T=5, B=2, hq=4, hk=2, d=128, out=E,
             ldo=512)
    a.update(kw)
    return sg.lib().ptpc_attn_prompt(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"],
                                     a["cu"], a["T"], a["B"], a["hq"], a["hk"], a["d"], 0.1,
                                     a["out"], a["ldo"], None)


FP8 = dict(fp8=1, dk=A, dv=B)


@pytest.mark.parametrize("call", [append, paged])
def test_cache_refusals(call):
    assert call() == HIP
    assert call(cache(**FP8)) == HIP
    assert call(cache(pages=-1)) == SHAPE
    assert call(cache(heads=-2)) == SHAPE
    for bad in (dict(page=8), dict(page=24), dict(page=1 << 17), dict(page=0), dict(d=96),
                dict(d=0), dict(heads=0), dict(heads=5000), dict(pages=1 << 31), dict(fp8=2)):
        assert call(cache(**bad)) == UNSUPPORTED, bad
    assert call(cache(k=None)) == NULLP
    assert call(cache(v=None)) == NULLP
    assert call(cache(fp8=1, dk=A)) == NULLP
    assert call(cache(k=MIS)) == ALIGN
    assert call(cache(fp8=1, dk=MIS, dv=B)) == ALIGN


def test_append_refusals():
    assert append(T=0) == OK
    assert append(cache(pages=0, k=None, v=None)) == HIP          # nothing to store, q still turns
    assert append(hq=0, q=None, out=None, ldq=0, ldqo=0) == HIP
    assert append(rot=0, table=None) == HIP
    for bad in (dict(T=-1), dict(hq=-1), dict(rot=-16), dict(rot=144), dict(n_pos=-1),
                dict(ldk=248), dict(ldv=248), dict(ldq=504), dict(ldqo=504)):
        assert append(**bad) == SHAPE, bad
    for bad in (dict(rot=24), dict(T=(1 << 24) + 1), dict(hq=4097), dict(ldk=(1 << 22) + 8),
                dict(ldqo=(1 << 22) + 8), dict(T=1 << 24, hq=16, ldq=2048, ldqo=2048)):
        assert append(**bad) == UNSUPPORTED, bad
    for bad in ("q", "k", "v", "table", "pos", "slots", "out"):
        assert append(**{bad: None}) == NULLP, bad
    for bad in (dict(q=MIS), dict(k=MIS), dict(v=MIS), dict(out=MIS), dict(table=MIS),
                dict(ldq=516), dict(ldk=260), dict(ldv=260), dict(ldqo=516), dict(pos=0x10002),
                dict(slots=0x10004)):
        assert append(**bad) == ALIGN, bad
    assert sg.lib().ptpc_rope_append(*([None, 0] * 3), None, 0, 0, 0, None, None, 0, 0, None,
                                     None, 0, None) == NULLP


def test_paged_refusals():
    assert paged(T=0) == OK and paged(B=0) == OK
    assert paged(width=0, ldt=0, table=None) == HIP
    assert paged(max_q=0, max_kv=0, ws=None, nb=0) == HIP
    for bad in (dict(T=-1), dict(B=-1), dict(hq=-4), dict(ldq=504), dict(ldo=504), dict(ldt=7),
                dict(max_q=-1), dict(max_kv=-1), dict(width=-1)):
        assert paged(**bad) == SHAPE, bad
    for bad in (dict(hq=3), dict(hq=0), dict(hq=4098), dict(T=(1 << 24) + 1),
                dict(B=(1 << 24) + 1), dict(ldq=(1 << 22) + 8), dict(max_kv=1 << 31),
                dict(max_kv=(1 << 30) + 1), dict(B=(1 << 19) + 1), dict(T=1 << 24, hq=32, ldq=4096,
                                                                      ldo=4096)):
        assert paged(**bad) == UNSUPPORTED, bad
    for bad in ("q", "cu", "table", "lens", "out"):
        assert paged(**{bad: None}) == NULLP, bad
    for bad in (dict(q=MIS), dict(out=MIS), dict(ldq=516), dict(ldo=516), dict(cu=0x10002),
                dict(lens=0x10001), dict(table=0x10002)):
        assert paged(**bad) == ALIGN, bad


def test_paged_workspace():
    f = sg.lib().ptpc_attn_paged_workspace_bytes
    for bad in (dict(T=0), dict(B=0), dict(max_q=0), dict(max_kv=0), dict(hq=3), dict(hq=0)):
        a = dict(T=1, B=1, max_q=1, max_kv=30000, hq=4)
        a.update(bad)
        assert f(a["T"], a["B"], a["max_q"], a["max_kv"], a["hq"], cache()) == 0, bad
    assert f(1, 1, 1, 30000, 4, cache(page=24)) == 0
    assert f(1, 1, 1, 30000, 4, None) == 0
    need = f(1, 1, 1, 30000, 4, cache())
    assert need > 0                               # one row over many keys: split
    one = dict(T=1, B=1, max_q=1, max_kv=30000)
    assert paged(**one, nb=need) == HIP
    assert paged(**one, nb=need - 1) == SHAPE
    assert paged(**one, ws=None) == NULLP
    assert paged(**one, ws=MIS) == ALIGN


def test_prompt_refusals():
    assert prompt() == HIP
    assert prompt(T=0) == OK and prompt(B=0) == OK
    for bad in (dict(T=-1), dict(B=-1), dict(hk=-1), dict(d=-64), dict(ldq=504), dict(ldk=248),
                dict(ldv=248), dict(ldo=504)):
        assert prompt(**bad) == SHAPE, bad
    for bad in (dict(d=96), dict(hq=3), dict(hk=0), dict(T=(1 << 24) + 1), dict(hq=8192, hk=1),
                dict(ldk=(1 << 22) + 8), dict(ldv=(1 << 22) + 8)):
        assert prompt(**bad) == UNSUPPORTED, bad
    for bad in ("q", "k", "v", "cu", "out"):
        assert prompt(**{bad: None}) == NULLP, bad
    for bad in (dict(q=MIS), dict(k=MIS), dict(v=MIS), dict(out=MIS), dict(ldq=516),
                dict(ldk=260), dict(ldv=260), dict(ldo=516), dict(cu=0x10002)):
        assert prompt(**bad) == ALIGN, bad


# ---- the binding ---------------------------------------------------------------------

class NoCompute:
    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*a):
            raise AssertionError(f"{name} was called with a mismatched argument")
        return call


@pytest.fixture
def cpu_binding(monkeypatch):
    monkeypatch.setattr(sg, "_lib", NoCompute(sg.lib()))
    monkeypatch.setattr(sg, "_on_gpu", lambda t, name: None)


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def raises(fn, match):
    with pytest.raises((ValueError, TypeError), match=match):
        fn()


def test_binding_cache(cpu_binding):
    k = bf(3, 2, 16, 64)
    u = torch.zeros((3, 2, 16, 64), dtype=torch.uint8)
    s = torch.zeros((3, 2, 16))
    sg.KVCache(k, k.clone())
    c = sg.KVCache(u, u.clone(), s, s.clone())
    assert (c.pages, c.kv_heads, c.page_size, c.head_dim, c.fp8) == (3, 2, 16, 64, True)
    raises(lambda: sg.KVCache(k.float(), k), "k: expected")
    raises(lambda: sg.KVCache(k, u), "v: expected")
    raises(lambda: sg.KVCache(k[0], k[0]), "k: expected")
    raises(lambda: sg.KVCache(k, k[:2]), "v: expected shape")
    raises(lambda: sg.KVCache(k, k.transpose(1, 2).contiguous().transpose(1, 2)), "contiguous")
    raises(lambda: sg.KVCache(u, u), "dk, dv")
    raises(lambda: sg.KVCache(k, k, s, s), "dk, dv")
    raises(lambda: sg.KVCache(u, u, s, s[:2]), "dv: expected shape")
    raises(lambda: sg.KVCache(u, u, s, s.double()), "dv: expected")
    with pytest.raises(AttributeError):
        c.k = k


def test_binding_append(cpu_binding):
    c = sg.KVCache(bf(3, 2, 16, 64), bf(3, 2, 16, 64))
    q, k, tab, pos, slots = bf(5, 4, 64), bf(5, 2, 64), torch.zeros(9, 64), i32(5), i32(5).long()
    f = sg.rope_append
    raises(lambda: f(q.float(), k, k, tab, pos, slots, c), "q: expected")
    raises(lambda: f(q[0], k, k, tab, pos, slots, c), "q: expected")
    raises(lambda: f(bf(5, 4, 128), k, k, tab, pos, slots, c), "q: expected shape")
    raises(lambda: f(bf(4, 5, 64).transpose(0, 1), k, k, tab, pos, slots, c), "one after another")
    raises(lambda: f(q, k[:4], k, tab, pos, slots, c), "k: expected shape")
    raises(lambda: f(q, k, q, tab, pos, slots, c), "v: expected shape")
    raises(lambda: f(q, k, k, tab.half(), pos, slots, c), "table: expected")
    raises(lambda: f(q, k, k, tab[0], pos, slots, c), "table: expected")
    raises(lambda: f(q, k, k, tab[:, :32], pos, slots, c), "table: expected")
    raises(lambda: f(q, k, k, tab, pos.long(), slots, c), "positions: expected")
    raises(lambda: f(q, k, k, tab, pos[:4], slots, c), "positions: expected")
    raises(lambda: f(q, k, k, tab, pos, pos, c), "slots: expected")
    raises(lambda: f(q, k, k, tab, pos, slots, c, q_out=bf(5, 3, 64)), "q_out: expected shape")


def test_binding_paged(cpu_binding):
    c = sg.KVCache(bf(3, 2, 16, 64), bf(3, 2, 16, 64))
    q, cu, tab, lens = bf(5, 4, 64), i32(3), i32(2, 6), i32(2)
    f = sg.attn_paged
    raises(lambda: f(bf(5, 4, 128), cu, c, tab, lens), "q: expected shape")
    raises(lambda: f(q, i32(4), c, tab, lens), "cu_q: expected")
    raises(lambda: f(q, cu.long(), c, tab, lens), "cu_q: expected")
    raises(lambda: f(q, cu, c, tab, lens.long()), "kv_lens: expected")
    raises(lambda: f(q, cu, c, tab, i32(2, 1)), "kv_lens: expected")
    raises(lambda: f(q, cu, c, tab.long(), lens), "page_table: expected")
    raises(lambda: f(q, cu, c, i32(3, 6), lens), "page_table: expected")
    raises(lambda: f(q, cu, c, i32(6, 2).t(), lens), "page_table: expected")
    raises(lambda: f(q, cu, c, tab, lens, out=bf(5, 2, 64)), "out: expected shape")
    raises(lambda: f(q, cu, c, tab, lens, max_kv=30000,
                     workspace=torch.zeros(16, dtype=torch.uint8)), "workspace: expected at least")


def test_binding_prompt(cpu_binding):
    q, k, cu = bf(5, 4, 64), bf(5, 2, 64), i32(3)
    f = sg.attn_prompt
    raises(lambda: f(q, k, bf(5, 1, 64), cu), "v: expected shape")
    raises(lambda: f(q, bf(4, 2, 64), k, cu), "k: expected shape")
    raises(lambda: f(q, bf(5, 2, 128), k, cu), "k: expected shape")
    raises(lambda: f(q.half(), k, k, cu), "q: expected")
    raises(lambda: f(q, k, k, cu.long()), "cu: expected")
    raises(lambda: f(q, k, k, i32(0)), "cu: expected")
    raises(lambda: f(q, k, k, cu, out=q[:4]), "out: expected shape")


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="on the GPU"):
        sg.KVCache(bf(3, 2, 16, 64), bf(3, 2, 16, 64))
    with pytest.raises(ValueError, match="on the GPU"):
        sg.attn_prompt(bf(5, 4, 64), bf(5, 2, 64), bf(5, 2, 64), i32(3))


# ---- the host layer under sanitizers ----------------------------------------------------

@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the ROCm headers not available")
def test_host_layer_under_sanitizers(tmp_path):
    exe = str(tmp_path / "attn_fuzz")
    csrc = os.path.join(ROOT, "scaled_gemm_amd", "csrc")
    cmd = ["g++", "-std=c++20", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g",
           "-O1", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(ROOT, "tests", "sanitize", "attn_fuzz.cpp"),
           os.path.join(csrc, "attn_api.cpp"), os.path.join(csrc, "attn_plan.cpp"), "-o", exe]
    for c in (cmd, [exe]):
        env = {k: v for k, v in os.environ.items() if k != "PTPC_FAULT"}
        r = subprocess.run(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, env=env)
        assert r.returncode == 0, r.stdout[-4000:]
    assert " 0 failures" in r.stdout, r.stdout


def test_struct_matches_the_header():
    text = open(os.path.join(ROOT, "include", "ptpc.h")).read()
    body = text[text.index("typedef struct {\n    void* k;"):text.index("} ptpc_kv_cache;")]
    names = [w.strip("; ") for w in body.split() if w.endswith(";")]
    assert names == [f[0] for f in sg._CacheStruct._fields_]
    assert ctypes.sizeof(sg._CacheStruct) == 72


def test_bound_of_the_gpu_tests():
    """The unit roundoff the attention bound is derived with is bf16's."""
    import attention_ref as ref
    assert ref.U / 2 < ref.bf16_roundoff() <= ref.U
