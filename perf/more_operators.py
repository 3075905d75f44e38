"""Cases of the block-scaled FP8 operators and the experts: what is measured, and their plain forms.

Five operators of a decoder layer's feed-forward half:

  quant     activations to E4M3 codes with one fp32 scale per token and block of 128
            channels; gated: of silu(first half) * second half;
  gemm      the FP8 product of such activations with a weight that has one scale per
            block of 128 x 128;
  route     softmax or sigmoid scores of the experts, a bias for balance, groups, the
            top k with their weights, and the (token, choice) pairs sorted by expert;
  experts   that product for every pair with its expert's weight, rows sorted by expert
            (gather: the rows are read from the tokens' activations);
  combine   each token's weighted sum of its experts' rows.

With `own` false, `run` computes them from elementary torch operations (32 bits; the
scores that decide between experts in 64); with `own` true it calls the framework.
The dense layers have the sizes of the 70B shaped projections or generic ones, with
blocks that the sizes do not fill among them.
"""
import math

import torch

own = False

BLOCK = 128


def listed():
    return [
        # one decode step's activations before a projection: the call is all latency
        dict(name="quant_step", op="quant", T=32, C=4096, gate=False),
        # a prompt's rows between an expert layer's two products, an odd number of them
        dict(name="quant_gate_prompt", op="quant", T=24577, C=1408, gate=True),
        # one token through a QKV projection: a stream of the weight
        dict(name="gemm_one", op="gemm", T=1, Ci=8192, Co=10240),
        # an odd chunk through an odd layer, the last block of each side partly filled
        dict(name="gemm_odd", op="gemm", T=333, Ci=2736, Co=4112),
        # a full prompt through a down projection
        dict(name="gemm_prompt", op="gemm", T=8192, Ci=28672, Co=8192),
        # a small decode batch: 256 experts in 8 groups, sigmoid scores with a balance bias
        dict(name="route_step", op="route", T=16, E=256, K=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, bf16=False),
        # a prompt's tokens: softmax over 128 experts, bf16 logits (equal ones among them)
        dict(name="route_prompt", op="route", T=8192, E=128, K=8, score="softmax", bias=False,
             groups=1, top_groups=1, bf16=True),
        # a few tokens in decode: some of 64 small experts, one or two rows each
        dict(name="experts_few", op="experts", T=4, E=64, K=6, Ci=2048, Co=2816, gather=True),
        # a decode batch's second product: 128 experts, about sixteen rows each
        dict(name="experts_step_down", op="experts", T=256, E=128, K=8, Ci=1408, Co=4096,
             gather=False),
        # a prompt's first product: hundreds of rows for each of 64 experts, gathered
        dict(name="experts_prompt", op="experts", T=4096, E=64, K=6, Ci=2048, Co=2816, gather=True),
        # one decode step's sum over eight experts
        dict(name="combine_step", op="combine", T=16, K=8, C=4096),
        # a prompt's
        dict(name="combine_prompt", op="combine", T=8191, K=8, C=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi):
    """A channel count: whole blocks mostly, else a multiple of 16."""
    step = rng.choice([128, 128, 16])
    return max(step, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "route", "experts", "experts", "combine"])
    T = _log(rng, 1, 8192)
    if op == "quant":
        return dict(op=op, T=T, C=_wide(rng, 512, 8192), gate=rng.random() < 0.5)
    if op == "gemm":
        return dict(op=op, T=T, Ci=_wide(rng, 512, 16384), Co=_wide(rng, 512, 12288))
    if op == "combine":
        return dict(op=op, T=T, K=rng.randint(1, 8), C=_wide(rng, 512, 4096))
    E = rng.choice([8, 16, 60, 64, 128, 256])
    K = rng.choice([1, 2, 4, 6, 8])
    if op == "route":
        groups = rng.choice([1, 1, 4])
        return dict(op=op, T=T, E=E, K=K, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups,
                    top_groups=groups if groups == 1 or K > E // 2 else 2, bf16=rng.random() < 0.5)
    Ci, Co = _wide(rng, 512, 4096), _wide(rng, 512, 4096)
    E = min(E, max(8, (1 << 30) // (Ci * Co)))
    return dict(op=op, T=max(1, min(T, (1 << 38) // (K * Ci * Co))), E=E, K=K, Ci=Ci, Co=Co,
                gather=rng.random() < 0.5)


def _blocks(n):
    return -(-n // BLOCK)


# ---- inputs ------------------------------------------------------------------------

def _codes(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _weight(shape, g):
    """Codes [.., Ci, Co] and scales [.., blocks of Ci, blocks of Co] of a weight whose blocks
    differ in size, as a checkpoint holds them."""
    *lead, ci, co = shape
    kb, nb = _blocks(ci), _blocks(co)
    n = math.prod(lead)
    codes = torch.empty((n, ci, co), dtype=torch.uint8, device="cuda")
    scales = 0.02 / 448 * torch.exp(0.3 * torch.randn((n, kb, nb), device="cuda", generator=g))
    for e in range(n):
        codes[e] = _codes((140.0 * torch.randn((ci, co), device="cuda", generator=g)).clamp_(-448, 448))
    return codes.view(*shape), scales.view(*lead, kb, nb)


def _acts(T, C, g):
    """bf16 activations: a few channels far larger than the rest, and rows of different size."""
    x = torch.randn((T, C), device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn((T, 1), device="cuda", generator=g))
    x *= torch.where(torch.rand(C, device="cuda", generator=g) < 0.01, 30.0, 1.0)
    return x.bfloat16()


def _logits(T, E, g):
    """Router logits: some experts are asked for more often than others."""
    x = torch.randn((T, E), device="cuda", generator=g)
    return x + 0.5 * torch.randn(E, device="cuda", generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T = case["op"], case["T"]
    st = dict(case=case)
    if op == "quant":
        st["x"] = _acts(T, case["C"] * (2 if case["gate"] else 1), g)
        if case["gate"]:
            st["x"][:, :case["C"]].clamp_(-20, 20)
    elif op == "gemm":
        st["qx"], st["sx"] = _quantized(_acts(T, case["Ci"], g).float())
        st["qw"], st["sw"] = _weight((case["Ci"], case["Co"]), g)
    elif op == "route":
        x = _logits(T, case["E"], g)
        st["logits"] = x.bfloat16() if case["bf16"] else x
        st["bias"] = 0.05 * torch.randn(case["E"], device="cuda", generator=g) if case["bias"] else None
    else:
        E, K = case.get("E", 64), case["K"]
        r = _layout(torch.topk(_logits(T, E, g), K).indices.int(), E)
        r["weights"] = torch.rand((T, K), device="cuda", generator=g)
        r["weights"] /= r["weights"].sum(1, keepdim=True)
        st["routing"] = r
        if op == "combine":
            st["y"] = torch.randn((T * K, case["C"]), device="cuda", generator=g).bfloat16()
        else:
            st["qx"], st["sx"] = _quantized(_acts(T if case["gather"] else T * K, case["Ci"], g).float())
            st["qw"], st["sw"] = _weight((E, case["Ci"], case["Co"]), g)
            count = r["offsets"].diff()
            st["active"] = count.nonzero()[:, 0]           # the experts that have rows
            st["most"] = int(count.max().item())           # and the most rows of one
    if own:
        import scaled_gemm_amd as sg
        if "qw" in st:
            st["bw"] = sg.pack_weight_block(st["qw"], st["sw"])
        if "routing" in st:
            st["plan"] = sg.Routing(**st["routing"])
    return st


# ---- the passes ----------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if op == "quant":
        return (_own_quant if own else _plain_quant)(st)
    if op == "gemm":
        return (_own_gemm if own else _plain_gemm)(st)
    if op == "route":
        return (_own_route if own else _plain_route)(st)
    if op == "experts":
        return (_own_experts if own else _plain_experts)(st)
    return (_own_combine if own else _plain_combine)(st)


def _own_quant(st):
    import scaled_gemm_amd as sg
    qx, sx = sg.quant_act_block(st["x"], gate=st["case"]["gate"])
    return dict(qx=qx.view(torch.float8_e4m3fn), sx=sx)


def _own_gemm(st):
    import scaled_gemm_amd as sg
    return sg.gemm_block(st["qx"], st["sx"], st["bw"])


def _own_route(st):
    import scaled_gemm_amd as sg
    c = st["case"]
    r = sg.route_experts(st["logits"], c["K"], scoring=c["score"], bias=st["bias"],
                         groups=c["groups"], top_groups=c["top_groups"], scale=2.5)
    return dict(ids=r.ids, weights=r.weights, offsets=r.offsets, rows=r.rows, slots=r.slots)


def _own_experts(st):
    import scaled_gemm_amd as sg
    return sg.gemm_experts(st["qx"], st["sx"], st["bw"], st["plan"], gather=st["case"]["gather"])


def _own_combine(st):
    import scaled_gemm_amd as sg
    return sg.combine_experts(st["y"], st["plan"])


def _spread(s, n, dim):
    """Scales of blocks, one for each of n elements along dim."""
    return s.repeat_interleave(BLOCK, dim=dim).narrow(dim, 0, n)


def _quantized(x):
    """Codes [T, C] and scales [blocks of C, T] of fp32 x [T, C]."""
    T, C = x.shape
    kb = _blocks(C)
    y = torch.zeros((T, kb * BLOCK), device=x.device)
    y[:, :C] = x
    top = y.view(T, kb, BLOCK).abs().amax(-1)
    # (torch divides by a plain number by multiplying with its reciprocal)
    s = torch.where(top == 0, torch.ones_like(top), top / torch.full_like(top, 448.0))
    return _codes((x / _spread(s, C, 1)).clamp(-448, 448)), s.T.contiguous()


def _plain_quant(st):
    x = st["x"].float()
    if st["case"]["gate"]:
        a, b = x.chunk(2, dim=1)
        x = a / (1.0 + torch.exp(-a)) * b
    qx, sx = _quantized(x)
    return dict(qx=qx.view(torch.float8_e4m3fn), sx=sx)


def _rows32(qx, sx):
    return qx.view(torch.float8_e4m3fn).float() * _spread(sx.T, qx.shape[1], 1)


def _weight32(qw, sw):
    ci, co = qw.shape[-2:]
    return qw.view(torch.float8_e4m3fn).float() * _spread(_spread(sw, ci, -2), co, -1)


def _plain_gemm(st):
    return torch.matmul(_rows32(st["qx"], st["sx"]), _weight32(st["qw"], st["sw"])).bfloat16()


def _layout(ids, E):
    """The pairs (token, choice) sorted by expert, in their order within one."""
    flat = ids.flatten().long()
    rows = torch.sort(flat, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    slots = torch.empty_like(rows)
    slots[rows] = torch.arange(rows.numel(), device=ids.device)
    return dict(ids=ids, offsets=offsets, rows=rows.int(), slots=slots.view(ids.shape).int())


def _plain_route(st):
    c, x = st["case"], st["logits"].double()
    T, E = x.shape
    G, K = c["groups"], c["K"]
    if c["score"] == "softmax":
        s = torch.exp(x - x.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    choice = s if st["bias"] is None else s + st["bias"].double()
    if G > 1:
        best = choice.view(T, G, E // G).sort(-1, descending=True).values[:, :, :2].sum(-1)
        picked = best.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        allowed = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, picked, True)
        choice = choice.masked_fill(~allowed.repeat_interleave(E // G, dim=1), -math.inf)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :K]
    w = s.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * 2.5
    r = _layout(ids.int(), E)
    return dict(ids=r["ids"], weights=w.float(), offsets=r["offsets"], rows=r["rows"],
                slots=r["slots"])


def _plain_experts(st):
    r, c = st["routing"], st["case"]
    x = _rows32(st["qx"], st["sx"])
    if c["gather"]:
        x = x[r["rows"].long() // c["K"]]
    w = _weight32(st["qw"][st["active"]], st["sw"][st["active"]])
    at = torch.arange(x.shape[0], device=x.device)
    first = r["offsets"][:-1].long()[st["active"]]
    seg = torch.searchsorted(first, at, right=True) - 1      # which active expert a row has
    pos = at - first[seg]
    padded = torch.zeros((w.shape[0], st["most"], c["Ci"]), device=x.device)
    padded[seg, pos] = x
    return torch.bmm(padded, w)[seg, pos].bfloat16()


def _plain_combine(st):
    r = st["routing"]
    y = st["y"].float()[r["slots"].long()]
    return (y * r["weights"][..., None]).sum(1).bfloat16()


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op == "quant":
        C, n = case["C"], 2 if case["gate"] else 1
        return {"bytes": T * (2 * C * n + C + 4 * _blocks(C)), "flops": T * C * (2 + 4 * (n - 1))}
    if op == "route":
        e, k = case["E"], case["K"]
        return {"bytes": T * (e * (2 if case["bf16"] else 4) + 16 * k) + 4 * e + 4, "flops": 4 * T * e}
    if op == "combine":
        return {"bytes": T * (case["K"] * (2 * case["C"] + 8) + 2 * case["C"]),
                "flops": 2 * T * case["K"] * case["C"]}
    Ci, Co = case["Ci"], case["Co"]
    weight = Ci * Co + 4 * _blocks(Ci) * _blocks(Co)
    if op == "gemm":
        return {"bytes": T * (Ci + 4 * _blocks(Ci) + 2 * Co) + weight, "flops": 2 * T * Ci * Co}
    E, K = case["E"], case["K"]
    active = E * (1.0 - (1.0 - K / E) ** T)
    rows = T if case["gather"] else T * K
    return {"bytes": int(active * weight) + rows * (Ci + 4 * _blocks(Ci)) + T * K * (2 * Co + 4),
            "flops": 2 * T * K * Ci * Co}


# ---- the definitions in 64 bits ----------------------------------------------------------

def _e4m3_64(x):
    """x (64 bits) rounded to the nearest E4M3 value, ties to even, at most 448 in magnitude."""
    _, e = torch.frexp(x)
    ulp = torch.ldexp(torch.ones_like(x), (e - 1).clamp_min(-6) - 3)
    return (torch.round(x / ulp) * ulp).clamp(-448.0, 448.0)


def _product64(qx, sx, qw, sw):
    """Block by block along the sum: each block's product, scaled on both sides."""
    total = torch.zeros((qx.shape[0], qw.shape[1]), dtype=torch.float64, device=qx.device)
    columns = torch.arange(qw.shape[1], device=qx.device) // BLOCK
    for b in range(sx.shape[0]):
        k = slice(b * BLOCK, (b + 1) * BLOCK)
        p = qx[:, k].view(torch.float8_e4m3fn).to(torch.float64) @ qw[k].view(torch.float8_e4m3fn).to(torch.float64)
        total += p * sx[b].double()[:, None] * sw[b].double()[columns]
    return total


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        x = st["x"].double()
        C = case["C"]
        if case["gate"]:
            x = x[:, :C] * torch.sigmoid(x[:, :C]) * x[:, C:]
        q, s = torch.empty_like(x), []
        for a in range(0, C, BLOCK):
            top = x[:, a:a + BLOCK].abs().amax(1)
            s.append(torch.where(top == 0, 1.0, top / 448.0))
            q[:, a:a + BLOCK] = _e4m3_64(x[:, a:a + BLOCK] / s[-1][:, None])
        return dict(qx=q, sx=torch.stack(s))
    if op == "gemm":
        return _product64(st["qx"], st["sx"], st["qw"], st["sw"])
    if op == "route":
        x = st["logits"].double()
        s = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
        c = s.cpu().numpy() + (0.0 if st["bias"] is None else st["bias"].double().cpu().numpy())
        E, G, K = case["E"], case["groups"], case["K"]
        import numpy as np
        if G > 1:
            best = np.sort(c.reshape(-1, G, E // G), axis=2)[:, :, -2:].sum(2)
            keep = np.argsort(-best, axis=1, kind="stable")[:, :case["top_groups"]]
            mask = np.ones((c.shape[0], G), dtype=bool)
            np.put_along_axis(mask, keep, False, axis=1)
            c = np.where(np.repeat(mask, E // G, axis=1), -np.inf, c)
        ids = np.argsort(-c, axis=1, kind="stable")[:, :K]
        w = np.take_along_axis(s.cpu().numpy(), ids, axis=1)
        order = np.argsort(ids.reshape(-1), kind="stable")
        slots = np.empty_like(order)
        slots[order] = np.arange(order.size)
        offsets = np.searchsorted(ids.reshape(-1)[order], np.arange(E + 1))
        whole = [torch.from_numpy(v.astype(np.int32)) for v in
                 (ids, offsets, order, slots.reshape(ids.shape))]
        return dict(ids=whole[0], weights=torch.from_numpy(2.5 * w / w.sum(1, keepdims=True)),
                    offsets=whole[1], rows=whole[2], slots=whole[3])
    r = st["routing"]
    if op == "combine":
        out = torch.zeros((case["T"], case["C"]), dtype=torch.float64, device="cuda")
        for k in range(case["K"]):
            out += st["y"][r["slots"][:, k].long()].double() * r["weights"][:, k, None].double()
        return out
    out = torch.empty((case["T"] * case["K"], case["Co"]), dtype=torch.float64, device="cuda")
    at = r["offsets"].tolist()
    for e in range(case["E"]):
        if at[e + 1] > at[e]:
            rows = torch.arange(at[e], at[e + 1], device="cuda")
            if case["gather"]:
                rows = r["rows"][rows].long() // case["K"]
            out[at[e]:at[e + 1]] = _product64(st["qx"][rows], st["sx"][:, rows], st["qw"][e], st["sw"][e])
    return out
