"""Operators between a layer's q, k, v products and its output product: rotary positions with the paged
key-value cache, and the attentions that read the cache.

The cache is k, v [pages][kv heads][page][D], bf16, or e4m3 with one fp32 scale per kv head; slot number
i is offset i % page of page i / page.  A sequence's tokens are in the pages that its row of the table
names, in order.

``run`` computes the plain forms (elementary torch operations in 32 bits, angles in 64), or, where ``own``
is true, makes the framework's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
CACHES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of an 8B layer, q, k, v as the decode products leave them: the smallest call
        {"name": "rope 1 token", "op": "rope", "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "type": "fp32", "norm": True,
         "inter": False, "cache": "bf16", "page": 64, "far": 4096, "prompt": False},
        # a decode batch at far positions, a quarter of the head rotated, into 8-bit pages
        {"name": "rope 61 tokens e4m3", "op": "rope", "T": 61, "Hq": 40, "Hkv": 8, "D": 128, "R": 32, "type": "bf16",
         "norm": False, "inter": True, "cache": "e4m3", "page": 16, "far": 1000000, "prompt": False},
        # a long prompt of a 14B layer
        {"name": "rope 8192 tokens", "op": "rope", "T": 8192, "Hq": 40, "Hkv": 8, "D": 128, "R": 128, "type": "fp32",
         "norm": True, "inter": False, "cache": "bf16", "page": 64, "far": 32768, "prompt": True},
        # one request that has just begun to answer: the smallest decode call
        {"name": "decode 1 short", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "len": 500, "cache": "bf16", "page": 64},
        # one request with a very long context, 14B heads: the split over the cache's length
        {"name": "decode 1 long", "op": "decode", "B": 1, "Hq": 40, "Hkv": 8, "D": 128, "len": 131072, "cache": "bf16", "page": 64},
        # a full decode batch, contexts from none to long
        {"name": "decode 64 ragged", "op": "decode", "B": 64, "Hq": 32, "Hkv": 8, "D": 128, "len": 8192, "cache": "bf16", "page": 16},
        # a decode batch on an 8-bit cache
        {"name": "decode 16 e4m3", "op": "decode", "B": 16, "Hq": 32, "Hkv": 8, "D": 128, "len": 32768, "cache": "e4m3", "page": 64},
        # heads of 64 in odd groups, an odd batch
        {"name": "decode 33 heads of 64", "op": "decode", "B": 33, "Hq": 14, "Hkv": 2, "D": 64, "len": 5000, "cache": "bf16", "page": 32},
        # a short prompt
        {"name": "prompt 200", "op": "prompt", "T": 200, "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "before": 0, "cache": "bf16", "page": 64},
        # packed prompts of many lengths
        {"name": "prompt 13 packed", "op": "prompt", "T": 8001, "B": 13, "Hq": 32, "Hkv": 8, "D": 128, "before": 0, "cache": "bf16", "page": 16},
        # one long prompt
        {"name": "prompt 8192", "op": "prompt", "T": 8192, "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "before": 0, "cache": "bf16", "page": 64},
        # the next chunk of a prompt whose beginning is in an 8-bit cache
        {"name": "prompt chunk e4m3", "op": "prompt", "T": 257, "B": 1, "Hq": 40, "Hkv": 8, "D": 128, "before": 32000,
         "cache": "e4m3", "page": 32},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "decode", "decode", "prompt", "prompt", "prompt"])
    Hkv = rng.choice([1, 2, 4, 8])
    c = {"op": op, "Hkv": Hkv, "Hq": Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]) if Hkv < 8 else Hkv * rng.choice([1, 2, 4, 5]),
         "D": rng.choice([64, 128, 128]), "cache": rng.choice(["bf16", "bf16", "e4m3"]), "page": rng.choice([16, 32, 64, 128])}
    if op == "rope":
        D = c["D"]
        return {**c, "T": _size(rng, 1, 8192), "R": rng.choice([D, D, D // 2, D // 4, D // 2 + 2]), "type": rng.choice(sorted(TYPES)),
                "norm": rng.random() < 0.5, "inter": rng.random() < 0.5, "far": _size(rng, 8192, 1000000), "prompt": rng.random() < 0.5}
    if op == "decode":
        B = _size(rng, 1, 128)
        return {**c, "B": B, "len": _size(rng, 1, min(65536, 524288 // B))}
    T = _size(rng, 1, 6000)
    B = _size(rng, 1, min(16, T))
    return {**c, "T": T, "B": B, "before": rng.choice([0, 0, _size(rng, 1, 8192)]) if T <= 2048 else 0}


# ---------------------------------------------------------------- lengths of a case (the seed only shuffles them)
def _lengths(case):
    """(new tokens, tokens in the cache with the new ones) of every sequence: lists of B."""
    B = case["B"]
    if case["op"] == "decode":  # from nothing (a padded row of the batch) to the longest
        if B == 1:
            return [1], [case["len"]]
        lens = [int(case["len"] ** (b / (B - 1))) for b in range(B)]
        lens[0] = 0
        return [1] * B, lens
    share = [1 + 2 * b for b in range(B)]  # packed prompts: the longest is about twice the average
    new = [case["T"] * s // sum(share) for s in share]
    new[-1] += case["T"] - sum(new)
    before = [case["before"] * (b + 1) // B for b in range(B)]
    return new, [n + p for n, p in zip(new, before)]


def _frequencies(case):
    """Angles a position, the slow ones stretched four times: fp32 [R/2]."""
    R = case["R"]
    f = 1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    return torch.where(f * 32768 > 2 * math.pi, f, f / 4).float()


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    mix = random.Random(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    Hq, Hkv, D, page = (case[n] for n in ("Hq", "Hkv", "D", "page"))
    st = {"case": case}
    if case["cache"] == "e4m3":
        st["k_scale"], st["v_scale"] = (0.01 + 0.01 * torch.rand(Hkv, generator=g, device=DEV) for _ in "kv")
    if case["op"] == "rope":
        T = case["T"]
        width = (Hq + 2 * Hkv) * D  # one row of the fused q, k, v product
        rows = (normal(T, width) * 1.5).to(TYPES[case["type"]])
        st["q"], st["k"], st["v"] = (x.unflatten(1, (-1, D)) for x in rows.split((Hq * D, Hkv * D, Hkv * D), 1))
        live = T - T // 16  # padded rows at the end
        pages = (live + page - 1) // page if case["prompt"] else live
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(T, device=DEV)
        if case["prompt"]:  # a prompt's tokens one after another, its pages anywhere
            st["positions"] = (mix.randrange(case["far"] - T + 1 if case["far"] > T else 1) + at).int()
            slots = order[at.clamp(max=live - 1) // page] * page + at % page
        else:  # every token of another sequence
            st["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=DEV).int()
            slots = order[at.clamp(max=live - 1)] * page + torch.randint(0, page, (T,), generator=g, device=DEV)
        st["slots"] = torch.where(at < live, slots, -1).int()
        st["freqs"] = _frequencies(case).to(DEV)
        if case["norm"]:
            st["q_norm"], st["k_norm"] = (1 + 0.1 * normal(D) for _ in "qk")
        st["cache_k"], st["cache_v"] = (torch.zeros(pages, Hkv, page, D, device=DEV).to(CACHES[case["cache"]]) for _ in "kv")
        return st
    new, lens = _lengths(case)
    order = list(range(case["B"]))
    mix.shuffle(order)
    new, lens = [new[b] for b in order], [lens[b] for b in order]
    most = max(1, max((n + page - 1) // page for n in lens))
    counts = [(n + page - 1) // page for n in lens]
    pages = sum(counts) + 1
    ids = torch.randperm(pages, generator=g, device=DEV).int().tolist()
    table = torch.full((case["B"], most), -1, dtype=torch.int32)
    for b, n in enumerate(counts):
        table[b, :n] = torch.tensor(ids[:n], dtype=torch.int32)
        ids = ids[n:]
    st["table"], st["lens"] = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["longest"] = max(lens)
    for n in ("k", "v"):
        scale = st[n + "_scale"].view(1, Hkv, 1, 1) if case["cache"] == "e4m3" else 1.0
        st["cache_" + n] = (normal(pages, Hkv, page, D) / scale).clamp(-448, 448).to(CACHES[case["cache"]])
    st["q"] = (normal(sum(new), Hq, D) * 1.5).to(torch.bfloat16)
    if case["op"] == "prompt":
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        st["most"] = max(new)
    return st


# ---------------------------------------------------------------- one pass, plainly
def _turn(x, cos, sin, R, inter):
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., : R // 2], x[..., R // 2 : R])
    turned = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack(turned, -1).flatten(-2) if inter else torch.cat(turned, -1)
    return torch.cat((turned, x[..., R:]), -1)


def _plain_rope(st):
    case = st["case"]
    angle = st["positions"].double()[:, None] * st["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    if case["norm"]:
        q = q / torch.sqrt((q * q).mean(-1, keepdim=True) + EPS) * st["q_norm"]
        k = k / torch.sqrt((k * k).mean(-1, keepdim=True) + EPS) * st["k_norm"]
    q, k = _turn(q, cos, sin, case["R"], case["inter"]), _turn(k, cos, sin, case["R"], case["inter"])
    if case["cache"] == "e4m3":
        k = (k / st["k_scale"][:, None]).clamp(-448, 448)
        v = (v / st["v_scale"][:, None]).clamp(-448, 448)
    at = (st["slots"] >= 0).nonzero(as_tuple=True)[0]
    slot = st["slots"][at].long()
    for cache, x in ((st["cache_k"], k), (st["cache_v"], v)):
        x = x[at].to(cache.dtype)
        if cache.dtype == torch.float8_e4m3fn:
            cache, x = cache.view(torch.uint8), x.view(torch.uint8)
        cache[slot // case["page"], :, slot % case["page"]] = x
    return {"q": q.to(torch.bfloat16), "k": st["cache_k"], "v": st["cache_v"]}


def _gather(st, name):
    """The first `longest` tokens of every sequence, fp32 [B, Hkv, longest, D] (past its end: page 0)."""
    page = st["case"]["page"]
    at = torch.arange(st["longest"], device=DEV)
    pages = st["table"].long().clamp(min=0)[:, at // page]
    cache = st["cache_" + name]
    if cache.dtype == torch.float8_e4m3fn:
        x = cache.view(torch.uint8)[pages, :, at % page].view(cache.dtype).float() * st[name + "_scale"][:, None]
    else:
        x = cache[pages, :, at % page].float()
    return x.transpose(1, 2)


def _attend(q, k, v, sees):
    """q [B, Hkv, rows, D], k and v [B, Hkv, L, D], sees [B, 1, rows, L]; rows that see nothing are 0."""
    s = torch.matmul(q * q.shape[-1] ** -0.5, k.transpose(2, 3)).masked_fill_(~sees, -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    return torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_attention(st):
    case = st["case"]
    B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    k, v, at, lens = _gather(st, "k"), _gather(st, "v"), torch.arange(st["longest"], device=DEV), st["lens"].long()
    if case["op"] == "decode":
        sees = (at < lens[:, None]).view(B, 1, 1, -1)
        return {"out": _attend(st["q"].float().view(B, Hkv, G, D), k, v, sees).reshape(B, Hq, D).to(torch.bfloat16)}
    starts, row = st["starts"].long(), torch.arange(st["most"], device=DEV)
    new = starts[1:] - starts[:-1]
    is_row = row < new[:, None]  # [B, most]
    q = torch.zeros(B, st["most"], Hkv, G, D, device=DEV)
    q[is_row] = st["q"].float().view(-1, Hkv, G, D)
    sees = at <= (lens - new)[:, None, None] + row[:, None]  # [B, most, L]
    y = _attend(q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D), k, v, sees.repeat(1, G, 1)[:, None])
    y = y.view(B, Hkv, G, -1, D).permute(0, 3, 1, 2, 4)[is_row]
    return {"out": y.reshape(-1, Hq, D).to(torch.bfloat16)}


def _own(st):
    from decode_gemv_thinkbit_amd import qlinear as ql

    case = st["case"]
    cache = ql.KvCache(st["cache_k"], st["cache_v"], st.get("k_scale"), st.get("v_scale"))
    if case["op"] == "rope":
        q = ql.rope_append(st["q"], st["k"], st["v"], st["positions"], st["slots"], ql.Rope(st["freqs"], interleaved=case["inter"]),
                           cache, q_norm=st.get("q_norm"), k_norm=st.get("k_norm"), eps=EPS)
        return {"q": q, "k": cache.k, "v": cache.v}
    if case["op"] == "decode":
        return {"out": ql.attn_decode(st["q"], cache, st["table"], st["lens"])}
    return {"out": ql.attn_prompt(st["q"], st["starts"], cache, st["table"], st["lens"])}


def run(state):
    if own:
        return _own(state)
    return _plain_rope(state) if state["case"]["op"] == "rope" else _plain_attention(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    Hq, Hkv, D = (case[n] for n in ("Hq", "Hkv", "D"))
    held = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "rope":
        T = case["T"]
        live = T - T // 16
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": T * (Hq * D * (size + 2) + 8) + live * 2 * Hkv * D * (size + held), "flops": T * (Hq + Hkv) * 3 * case["R"]}
    new, lens = _lengths(case)
    pairs = sum(n * (l - n) + n * (n + 1) // 2 for n, l in zip(new, lens) if l)
    return {"bytes": 2 * sum(lens) * Hkv * D * held + 4 * sum(new) * Hq * D + 4 * sum(-(-l // case["page"]) for l in lens),
            "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    Hq, Hkv, D, page = (case[n] for n in ("Hq", "Hkv", "D", "page"))
    if case["op"] == "rope":
        R = case["R"]
        pairs = torch.arange(R // 2, device=DEV)
        first, second = (2 * pairs, 2 * pairs + 1) if case["inter"] else (pairs, pairs + R // 2)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), st["positions"].double()[:, None, None] * st["freqs"].double())
        out = {}
        for n in "qk":
            x = st[n].double().clone()
            if case["norm"]:
                x = x * st[n + "_norm"].double() * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            out[n] = x
        out["v"] = st["v"].double()
        for n in "kv":
            cache = torch.zeros(st["cache_k"].shape, dtype=torch.float64, device=DEV).transpose(1, 2).flatten(0, 1)
            x = out[n] / st[n + "_scale"].double()[:, None] if case["cache"] == "e4m3" else out[n]
            live = st["slots"] >= 0
            cache[st["slots"][live].long()] = x[live].clamp(-448, 448) if case["cache"] == "e4m3" else x[live]
            out[n] = cache.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
        return out
    y = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    starts = st["starts"].tolist() if case["op"] == "prompt" else list(range(case["B"] + 1))
    G = Hq // Hkv
    for b, length in enumerate(st["lens"].tolist()):
        if not length:
            continue
        rows = st["table"][b, : -(-length // page)].long()
        kv = []
        for n in "kv":
            cache = st["cache_" + n]
            x = cache.view(torch.uint8)[rows].view(cache.dtype) if case["cache"] == "e4m3" else cache[rows]
            x = x.double().transpose(0, 1).flatten(1, 2)[:, :length]  # [Hkv, length, D]
            kv.append(x * st[n + "_scale"].double()[:, None, None] if case["cache"] == "e4m3" else x)
        k, v = kv
        n = starts[b + 1] - starts[b]
        for r0 in range(0, n, 1024):
            r1 = min(n, r0 + 1024)
            upto = length - n + r1  # what the last of these rows sees
            q = st["q"][starts[b] + r0 : starts[b] + r1].double().transpose(0, 1)  # [Hq, rows, D]
            late = torch.arange(upto, device=DEV)[None] > length - n + torch.arange(r0, r1, device=DEV)[:, None]
            for h in range(Hq):
                s = torch.mm(q[h], k[h // G, :upto].t()) / math.sqrt(D)
                s[late] = -math.inf
                y[starts[b] + r0 : starts[b] + r1, h] = torch.mm(torch.softmax(s, -1), v[h // G, :upto])
    return {"out": y}
