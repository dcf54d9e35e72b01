"""Operators on microscaled 4-bit floats (MX4) and the mixture-of-experts layer on them.

MX4: a value is e2m1(code) * 2^(s - 127); one byte s is shared by 32 consecutive inputs.  Codes are
[N][K/2] bytes (low nibble first), scales [N][4 * ceil(K/128)] bytes of which the first K/32 count.

``run`` computes the plain forms (elementary torch operations in 32 bits), or, where ``own`` is true,
makes the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode batch's activations before an MX4 x MX4 product
        {"name": "quantize activations", "op": "quantize", "rows": 16, "K": 4096, "type": "bf16"},
        # the largest linear of an 8B layer at load time
        {"name": "quantize weight", "op": "quantize", "rows": 12288, "K": 4096, "type": "fp32"},
        # one token through an attention projection of an 8B layer: the smallest decode call
        {"name": "gemv 1 token", "op": "gemv", "M": 1, "N": 4096, "K": 4096},
        # a full decode batch through the down projection of a 14B layer
        {"name": "gemv 16 tokens", "op": "gemv", "M": 16, "N": 5120, "K": 17408},
        # speculative tokens on a matrix whose rows and inputs end inside a tile
        {"name": "gemv ragged", "op": "gemv", "M": 5, "N": 1000, "K": 2080},
        # a large decode batch, ragged rows, through a 14B projection
        {"name": "gemm 33 tokens", "op": "gemm", "M": 33, "N": 5120, "K": 5120},
        # a prefill chunk through the up projection of an 8B layer
        {"name": "gemm 512 tokens", "op": "gemm", "M": 512, "N": 12288, "K": 4096},
        # a long prompt through the same
        {"name": "gemm 4096 tokens", "op": "gemm", "M": 4096, "N": 12288, "K": 4096},
        # the router of a decode batch, logits from a bf16 product (equal logits occur)
        {"name": "route 16 tokens", "op": "route", "T": 16, "E": 64, "k": 8, "type": "bf16", "renorm": True},
        # the router of a long prompt with padded rows
        {"name": "route 4096 tokens", "op": "route", "T": 4096, "E": 128, "k": 8, "type": "fp32", "renorm": False},
        # one decoded token through a layer of 64 experts
        {"name": "moe 1 token", "op": "moe", "T": 1, "E": 64, "k": 8, "H": 2048, "I": 1024, "renorm": True},
        # a decode batch through a layer of many small experts, sizes that end inside a tile
        {"name": "moe 24 tokens", "op": "moe", "T": 24, "E": 128, "k": 6, "H": 2080, "I": 736, "renorm": False},
    ]


def _size(rng, lo, hi, step=1):
    """A size spread over the logarithm of lo .. hi, a multiple of step."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "gemv", "gemv", "gemm", "gemm", "route", "moe", "moe"])
    if op == "quantize":
        return {"op": op, "rows": _size(rng, 1, 8192), "K": _size(rng, 32, 5120, 32), "type": rng.choice(sorted(TYPES))}
    if op == "gemv":
        return {"op": op, "M": rng.randint(1, 16), "N": _size(rng, 64, 12288), "K": _size(rng, 128, 12288, 32)}
    if op == "gemm":
        return {"op": op, "M": _size(rng, 1, 4096), "N": _size(rng, 64, 12288), "K": _size(rng, 128, 4096, 32)}
    E = _size(rng, 4, 128)
    k = rng.randint(1, min(E, 8))
    if op == "route":
        return {"op": op, "T": _size(rng, 1, 4096), "E": E, "k": k, "type": rng.choice(sorted(TYPES)),
                "renorm": rng.random() < 0.5}
    return {"op": op, "T": _size(rng, 1, 64), "E": E, "k": k, "H": _size(rng, 256, 2048, 32),
            "I": _size(rng, 128, 1024, 32), "renorm": rng.random() < 0.5}


# ---------------------------------------------------------------- the format, plainly
def _quantize(x):
    """Codes and scale exponents of x [..., K]: uint8 [..., K/2] and [..., 4 * ceil(K/128)]."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127).float()
    e = torch.where(top > 0, e, torch.full_like(e, -127.0))
    v = b / torch.exp2(e)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | ((v < 0).to(torch.uint8) << 3)).flatten(-2)
    s = (e.squeeze(-1) + 127).to(torch.uint8)
    s = torch.nn.functional.pad(s, (0, -s.shape[-1] % 4))
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def _values(codes, scales):
    """The fp32 values [..., K] of codes [..., K/2] and scales."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = table[c.int()].unflatten(-1, (-1, 32))
    s = scales[..., : v.shape[-2]].float() - 127
    return (v * torch.exp2(s).unsqueeze(-1)).flatten(-2)


def _route(logits, k, renorm):
    """The k largest of every row, the lowest index first among equals; -inf is never taken."""
    v = logits.float()
    top, ids = torch.sort(v, dim=-1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k].int()
    live = top > -math.inf
    most = top[:, :1].clamp(min=-3e38)
    w = torch.exp(top - most)
    w = w / (w if renorm else torch.exp(v - most)).sum(-1, keepdim=True).clamp(min=1e-30)
    return torch.where(live, ids, -1), torch.where(live, w, 0.0)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    op = case["op"]
    st = {"case": case}
    if op == "quantize":
        sigma = 0.02 if case["type"] == "fp32" else 1.0
        st["x"] = (normal(case["rows"], case["K"]) * sigma).to(TYPES[case["type"]])
    elif op == "gemv":
        st["w"] = _quantize(normal(case["N"], case["K"]) * 0.02)
        st["x"] = normal(case["M"], case["K"]).to(torch.bfloat16)
    elif op == "gemm":
        st["w"] = _quantize(normal(case["N"], case["K"]) * 0.02)
        st["x"] = _quantize(normal(case["M"], case["K"]))
    else:
        logits = normal(case["T"], case["E"]) * 1.5
        if op == "route":
            if case["T"] > 4:  # padded rows at the end, and experts masked here and there
                logits = logits.masked_fill(torch.rand(logits.shape, generator=g, device=DEV) < 0.02, -math.inf)
                logits[-(case["T"] // 8 + 1):] = -math.inf
            st["logits"] = logits.to(TYPES[case["type"]])
        else:
            T, E, H, I = (case[n] for n in "TEHI")
            st["logits"] = logits
            st["x"] = normal(T, H).to(torch.bfloat16)
            for name, rows, inner in (("gate", I, H), ("up", I, H), ("down", H, I)):
                st[name] = _quantize(normal(E, rows, inner) * 0.02)
    return st


# ---------------------------------------------------------------- one pass
def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        return {"values": _values(*_quantize(st["x"]))}
    if op == "gemv":
        return {"y": st["x"].float() @ _values(*st["w"]).t()}
    if op == "gemm":
        return {"y": _values(*st["x"]) @ _values(*st["w"]).t()}
    ids, weights = _route(st["logits"], case["k"], case["renorm"])
    out = {"ids": ids, "weights": weights}
    if op == "moe":
        x, pick, few = st["x"].float(), slice(None), case["T"] * case["k"] <= case["E"]
        if few:  # one expert's matrices for each (token, slot)
            pick = ids.long().clamp(min=0).flatten()
            x, scale = x.repeat_interleave(case["k"], 0).unsqueeze(1), weights.reshape(-1, 1, 1)
        else:  # every expert on every token, weight 0 where it was not picked
            dense = torch.zeros(case["T"], case["E"] + 1, device=x.device)
            scale = dense.scatter_add_(1, ids.long() % (case["E"] + 1), weights)[:, :-1].t().unsqueeze(-1)
        gate, up = (torch.matmul(x, _values(st[n][0][pick], st[n][1][pick]).transpose(1, 2)) for n in ("gate", "up"))
        h = gate / (1 + torch.exp(-gate)) * up * scale
        y = torch.matmul(h, _values(st["down"][0][pick], st["down"][1][pick]).transpose(1, 2))
        out["y"] = y.reshape(case["T"], -1, case["H"]).sum(1) if few else y.sum(0)
    return out


def _own(st):
    from decode_gemv_thinkbit_amd import qlinear as ql

    case = st["case"]
    op = case["op"]
    if op == "quantize":
        return {"values": ql.mx4_dequant(ql.mx4_quantize(st["x"]))}
    if op == "gemv":
        return {"y": ql.mx4_gemv(st["x"], ql.Mx4Tensor(*st["w"]))}
    if op == "gemm":
        return {"y": ql.mx4_gemm(ql.Mx4Tensor(*st["x"]), ql.Mx4Tensor(*st["w"]))}
    ids, weights = ql.moe_route(st["logits"], case["k"], renormalize=case["renorm"])
    out = {"ids": ids, "weights": weights}
    if op == "moe":
        out["y"] = ql.mx4_moe(st["x"], ids, weights, *(ql.Mx4Tensor(*st[n]) for n in ("gate", "up", "down")))
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": n * ((4 if case["type"] == "fp32" else 2) + 17 / 32 + 4), "flops": 3 * n}
    if op == "gemv":
        M, N, K = (case[n] for n in "MNK")
        return {"bytes": N * K * 17 / 32 + 2 * M * K + 4 * M * N, "flops": 2 * M * N * K}
    if op == "gemm":
        M, N, K = (case[n] for n in "MNK")
        return {"bytes": (M + N) * K * 17 / 32 + 4 * M * N, "flops": 2 * M * N * K}
    T, E, k = (case[n] for n in "TEk")
    if op == "route":
        return {"bytes": T * E * (4 if case["type"] == "fp32" else 2) + 8 * T * k, "flops": 4 * T * E}
    H, I = case["H"], case["I"]
    active = E * (1 - (1 - k / E) ** T)  # experts that some token picks, on average
    return {"bytes": active * 3 * I * H * 17 / 32 + 4 * T * E + 8 * T * k + 6 * T * H, "flops": 6 * T * k * I * H}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_block_values(x):
    """Every block's nearest MX4 values in fp64: the exponent from the largest value's own bits, each
    value by its distance to all eight magnitudes (those with even codes first, as ties go to them)."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    e = ((top.view(torch.int64) >> 52) - 1023 - 2).clamp(-127, 127)
    v = b * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), -e.double())
    grid = torch.tensor([0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0], dtype=torch.float64, device=x.device)
    best, far = torch.zeros_like(v), torch.full_like(v, math.inf)
    for m in grid:
        d = (v.abs() - m).abs()
        best, far = torch.where(d < far, m, best), torch.minimum(d, far)
    out = torch.copysign(best, v) * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), e.double())
    return out.reshape(x.shape)


def _exact_decode(codes, scales):
    c = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.int64, device=codes.device)
    c[..., 0::2], c[..., 1::2] = codes & 0x0F, codes >> 4
    m, ex, sign = c & 1, (c >> 1) & 3, c >> 3
    mag = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.pow(2.0, (ex - 1).double()))
    s = scales.to(torch.int64).repeat_interleave(32, -1)[..., : c.shape[-1]]
    return (1 - 2 * sign).double() * mag.double() * torch.pow(2.0, (s - 127).double())


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"values": _exact_block_values(st["x"])}
    if op in ("gemv", "gemm"):
        x = st["x"].double() if op == "gemv" else _exact_decode(*st["x"])
        return {"y": torch.matmul(x, _exact_decode(*st["w"]).t().contiguous())}
    T, E, k = (case[n] for n in "TEk")
    logits = st["logits"].double().cpu()
    ids, weights = torch.full((T, k), -1, dtype=torch.int32), torch.zeros(T, k, dtype=torch.float64)
    for t, row in enumerate(logits.tolist()):
        order = [e for e in sorted(range(E), key=lambda e: (-row[e], e)) if row[e] > -math.inf][:k]
        if order:
            over = sum(math.exp(row[e] - row[order[0]]) for e in (order if case["renorm"] else range(E)))
            for j, e in enumerate(order):
                ids[t, j], weights[t, j] = e, math.exp(row[e] - row[order[0]]) / over
    out = {"ids": ids, "weights": weights}
    if op == "moe":
        y = torch.zeros(T, case["H"], dtype=torch.float64, device=DEV)
        x = st["x"].double()
        for e in sorted(set(ids.flatten().tolist()) - {-1}):
            rows, slots = (ids == e).nonzero(as_tuple=True)
            rows = rows.to(DEV)
            gate, up, down = (_exact_decode(st[n][0][e], st[n][1][e]) for n in ("gate", "up", "down"))
            g = torch.matmul(x[rows], gate.t().contiguous())
            h = g * torch.sigmoid(g) * torch.matmul(x[rows], up.t().contiguous())
            w = weights[ids == e].to(DEV)
            y.index_add_(0, rows, torch.matmul(h, down.t().contiguous()) * w[:, None])
        out["y"] = y
    return out
