"""Plain 64-bit references of rotary positions, the paged cache and attention over it (CPU), the inputs of
their tests, and what the kernels' roundings may add up to."""
import math

import torch

EPS32 = 2.0 ** -24   # half a step of fp32, bf16, e4m3, relative to the value
EPS16 = 2.0 ** -8
EPS8 = 2.0 ** -4
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- rotary positions
def turned(x, positions, freqs, interleaved, factor, norm, eps):
    """x [T, heads, D] in 64 bits, normed and turned, and how far fp32 arithmetic may be from it."""
    x = x.double()
    T, _, D = x.shape
    rel = 0.0
    if norm is not None:
        x = x * norm.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        # the sum of D squares in any order, the mean, eps, root, quotient, two products: every factor of the result
        # is off by (1 + EPS32) at most, halved under the root
        rel = (D + 8) * EPS32
    R = 2 * freqs.numel()
    p = torch.arange(R // 2)
    first, second = (2 * p, 2 * p + 1) if interleaved else (p, p + R // 2)
    angle = positions.double()[:, None] * freqs.double()
    c, s = factor * torch.cos(angle)[:, None], factor * torch.sin(angle)[:, None]
    y = x.clone()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    # The angle's fraction is rounded to fp32 (pi 2^-24 radians at most), sine and cosine are within 4 steps of
    # 2^-24, two products, a sum and the factor add 4 more: 12 half steps of |u| + |v|
    size = x.abs().clone()
    size[..., first] = size[..., second] = (x[..., first].abs() + x[..., second].abs()) * abs(factor)
    return y, size * (rel + 12 * EPS32)


def bf16_close(got, want, slack):
    """bf16 within half a step of a value that is within slack of want (its steps end at 2^-133)."""
    return (got.double() - want).abs() <= slack + EPS16 * (want.abs() + slack) + 2.0 ** -134


def e4m3_close(got, want, slack):
    want = want.clamp(-448, 448)
    return (got.double() - want).abs() <= slack + EPS8 * (want.abs() + slack) + 2.0 ** -10


# ---------------------------------------------------------------- a cache of sequences
class Sequences:
    """Sequences of given lengths in a paged cache, pages in random order, and what is in them (64 bits)."""

    def __init__(self, lens, Hkv, D, page, cache="bf16", seed=0, spare=2, spread=1.0, fill=0.0, most=None):
        g = torch.Generator().manual_seed(seed)
        counts = [(max(n, 0) + page - 1) // page for n in lens]
        pages = sum(counts) + spare
        order = torch.randperm(pages, generator=g).int().tolist()
        self.most = max([1] + counts) if most is None else most
        self.table = torch.full((len(lens), self.most), -1, dtype=torch.int32)
        self.lens, self.page, self.Hkv, self.D = list(lens), page, Hkv, D
        dtype = F8 if cache == "e4m3" else torch.bfloat16
        self.scales = [torch.rand(Hkv, generator=g) * 0.02 + 0.01 for _ in "kv"] if cache == "e4m3" else [None, None]
        store = [torch.full((pages, Hkv, page, D), fill).to(dtype) for _ in "kv"]
        self.kv = []
        for b, (n, count) in enumerate(zip(lens, counts)):
            mine, order = order[:count], order[count:]
            self.table[b, :count] = torch.tensor(mine, dtype=torch.int32)
            both = []
            for z in range(2):
                x = torch.randn(max(n, 0), Hkv, D, generator=g) * spread
                if cache == "e4m3":
                    x = (x / self.scales[z][:, None]).clamp(-448, 448).to(dtype)
                    held = x.view(torch.uint8)
                    both.append(x.double() * self.scales[z].double()[:, None])
                else:
                    x = held = x.to(dtype)
                    both.append(x.double())
                to = store[z].view(torch.uint8) if cache == "e4m3" else store[z]
                for i, p in enumerate(mine):
                    part = held[i * page : (i + 1) * page]
                    to[p, :, : part.shape[0]] = part.transpose(0, 1)
            self.kv.append(both)
        self.k, self.v = store

    def on(self, dev):
        """(KvCache, table, lens) on the device."""
        from decode_gemv_thinkbit_amd import qlinear as ql

        s = [None if x is None else x.to(dev) for x in self.scales]
        return (ql.KvCache(self.k.to(dev), self.v.to(dev), *s), self.table.to(dev),
                torch.tensor(self.lens, dtype=torch.int32, device=dev))


def attention(q, k, v, sees, scale):
    """out [rows, Hq, D] in 64 bits of q [rows, Hq, D] over k, v [keys, Hkv, D], sees [rows, keys]; and the most that
    the kernels' roundings may move it."""
    rows, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, slack = torch.zeros(rows, Hq, D, dtype=torch.float64), torch.zeros(rows, Hq, D, dtype=torch.float64)
    if not k.shape[0]:
        return out, slack
    for h in range(Hq):
        qh, kh, vh = q[:, h].double(), k[:, h // G], v[:, h // G]
        s = (qh @ kh.t() * scale).masked_fill(~sees, -math.inf)
        top = s.amax(-1, keepdim=True).clamp(min=-1e300)
        w = torch.exp(s - top)
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
        w = torch.where(sees, w, 0.0)
        out[:, h] = w @ torch.nan_to_num(vh)
        size = w @ torch.nan_to_num(vh).abs()
        # A score is a sum of D products in fp32, scaled, and set off against the maximum: that moves a weight by the
        # factor exp(d).  exp2 is within 2 steps of fp32 and rounded to bf16, sums of up to n weights and values
        # are fp32, parts are joined with one more factor, and the quotient is one rounding.
        d = (D + 4) * EPS32 * scale * (qh.abs() @ torch.nan_to_num(kh).abs().t()).masked_fill(~sees, 0.0).amax(-1)
        d = d + 4 * EPS32 * torch.where(sees, s, 0.0).abs().amax(-1)
        n = sees.sum(-1).double()
        slack[:, h] = size * (EPS16 + 2 * torch.expm1(d) + 2 * (n + 12) * EPS32)[:, None]
    return out, slack


def decode(seqs, q, scale, visible=None):
    """attention() of one query a sequence: q [B, Hq, D]; visible: {b: bool [len]} of keys that count."""
    outs = []
    for b, (k, v) in enumerate(seqs.kv):
        sees = torch.ones(1, k.shape[0], dtype=torch.bool)
        if visible and b in visible:
            sees &= visible[b]
        outs.append(attention(q[b : b + 1], k, v, sees, scale))
    return torch.cat([o for o, _ in outs]), torch.cat([s for _, s in outs])


def prompt(seqs, q, starts, scale, visible=None):
    """attention() of packed queries: q [T, Hq, D]; rows of no sequence are 0."""
    out, slack = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for b, (k, v) in enumerate(seqs.kv):
        n, length = starts[b + 1] - starts[b], k.shape[0]
        if not n:
            continue
        sees = torch.arange(length)[None] <= length - n + torch.arange(n)[:, None]
        if visible and b in visible:
            sees &= visible[b]
        rows = slice(starts[b], starts[b + 1])
        out[rows], slack[rows] = attention(q[rows], k, v, sees, scale)
    return out, slack


def queries(rows, Hq, D, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, Hq, D, generator=g) * spread).to(torch.bfloat16)
