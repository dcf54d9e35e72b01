"""Calls of the rotary and attention operators that a program may make and the other tests do not: memory that moved, odd
strides of single rows, the ends of a type's range (GPU)."""
import pytest
import torch

import attn_reference as ref
from decode_gemv_thinkbit_amd import qlinear as ql

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ql.lib()
    return torch.device("cuda:0")


def ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_memory_that_moved(dev, kind):
    """A cache and frequencies whose tensors got other memory: it is read and written, what they had is not."""
    seqs = ref.Sequences([700, 30], 2, 64, 16, kind, seed=1)
    q = ref.queries(2, 4, 64, 2).to(dev)
    cache, table, lens = seqs.on(dev)
    rope = ql.Rope(torch.rand(32, generator=torch.Generator().manual_seed(3)).to(dev))
    starts = ints([0, 1, 2], dev)
    slots = ints([int(table[0, 0]) * 16, int(table[1, 0]) * 16 + 3], dev)
    rows = ref.queries(2, 2, 64, 4).to(dev)

    def calls():
        turned = ql.rope_append(q, rows, rows, ints([5, 9], dev), slots, rope, cache)
        return turned, ql.attn_decode(q, cache, table, lens), ql.attn_prompt(q, starts, cache, table, lens)

    want = [x.clone() for x in calls()]
    held = []
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, rope.freqs):
        if t is not None:
            old, fresh = t.detach(), t.clone()
            t.data = fresh
            (old.view(torch.uint8) if kind == "e4m3" and old.dtype == ref.F8 else old).fill_(0)
            held.append(old)
    got = calls()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((t.float() == 0).all() for t in held)


@pytest.mark.parametrize("new,before,front,behind,Hq,Hkv", [
    ([1] * 40, [(97 * b) % 5000 for b in range(40)], 0, 0, 8, 2), ([4] * 16, [1000 + 300 * b for b in range(16)], 0, 3, 8, 1),
    ([0, 5, 0, 130, 1], [9000, 3000, 0, 5000, 2], 7, 11, 4, 4), ([33, 40], [4000, 0], 2, 0, 6, 2), ([3], [20000], 0, 0, 40, 1)])
@pytest.mark.parametrize("D,kind", [(128, "bf16"), (64, "e4m3")])
def test_parts_of_prompts_stay_in_their_workspace(dev, new, before, front, behind, Hq, Hkv, D, kind):
    """Rows of many sequences in parts, a workspace of just the size that is asked for, full of NaN, memory around it kept."""
    seqs = ref.Sequences([n + p for n, p in zip(new, before)], Hkv, D, 16, kind, seed=len(new))
    starts = [front]
    for n in new:
        starts.append(starts[-1] + n)
    T, B = starts[-1] + behind, len(new)
    q = ref.queries(T, Hq, D, 5)
    cache, table, lens = seqs.on(dev)
    need = ql.lib().qlinear_attn_prompt_workspace_bytes(T, B, Hq, Hkv, D, 16 * seqs.most)
    assert need > 0
    buf = torch.full((need // 4 + 2048,), float("nan"), device=dev)
    ws = buf[1024 : 1024 + need // 4].view(torch.uint8)
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=dev)
    ql.attn_prompt(q.to(dev), ints(starts, dev), cache, table, lens, out=out, workspace=ws)
    want, slack = ref.prompt(seqs, q, starts, D ** -0.5)
    rows = slice(front, starts[-1])
    assert ref.bf16_close(out.cpu()[rows], want[rows], slack[rows]).all()
    assert (out[:front] == 5.0).all() and (out[starts[-1] :] == 5.0).all()
    assert torch.isnan(buf[:1024]).all() and torch.isnan(buf[-1024:]).all()


# ---------------------------------------------------------------- the ends of bf16's range
def of_size(seqs, exponent):
    """V positive, and 2^exponent times as large."""
    seqs.v = (seqs.v.float().abs() * 2.0 ** exponent).to(torch.bfloat16)
    for both in seqs.kv:
        both[1] = both[1].abs() * 2.0 ** exponent
    return seqs


def steps_below(n, lag):
    """What fp32's last step moves a result: n products and some 40 sums of parts are off by 2^-150 each, and the largest
    weight is 2^-room at least, with 2^room at most 4 n 2^lag."""
    return (n + 40) * 2.0 ** -150 * 4 * n * 2.0 ** lag


@pytest.mark.parametrize("lens", [[1], [2, 17, 500], [700, 3, 40], [9000]])
def test_decode_small_values(dev, lens):
    """V far below 1, where bf16 is still normal: nothing of it is lost among fp32's last steps but what they are."""
    seqs = of_size(ref.Sequences(lens, 2, 64, 16, seed=5), -112)
    q = ref.queries(len(lens), 4, 64, 6)
    want, slack = ref.decode(seqs, q, 64 ** -0.5)
    slack = slack + torch.tensor([steps_below(n, 0) for n in lens])[:, None, None]
    got = ql.attn_decode(q.to(dev), *seqs.on(dev)).cpu()
    assert ref.bf16_close(got, want, slack).all()


@pytest.mark.parametrize("n,length", [(1, 1), (20, 20), (300, 300), (700, 700), (5, 4000), (300, 4000)])
def test_prompt_small_values(dev, n, length):
    seqs = of_size(ref.Sequences([length], 2, 128, 16, seed=5), -112)
    q = ref.queries(n, 4, 128, 6)
    cache, table, lens = seqs.on(dev)
    got = ql.attn_prompt(q.to(dev), ints([0, n], dev), cache, table, lens).cpu()
    want, slack = ref.prompt(seqs, q, [0, n], 128 ** -0.5)
    assert ref.bf16_close(got, want, slack + steps_below(length, 8)).all()


@pytest.mark.parametrize("length", [1, 64, 127, 512, 513, 4095, 20000])
@pytest.mark.parametrize("exponent", [127, -118])
@pytest.mark.parametrize("lag", [0.0, 7.9])
def test_the_largest_sums_of_weights(dev, length, exponent, lag):
    """All of V one value, all keys but the first 64 weighing 2^lag times as much as those, which a maximum that follows
    only larger steps leaves as they are: the value comes out."""
    D, page = 64, 64
    pages = (length + page - 1) // page
    k = torch.zeros(pages, 1, page, D)
    k[1:, :, :, 0] = lag  # one score of q . k = lag, exact in the scale below
    k = k.to(torch.bfloat16)
    v = torch.full((pages, 1, page, D), 2.0 ** exponent).to(torch.bfloat16)
    cache = ql.KvCache(k.to(dev), v.to(dev))
    q = torch.zeros(3, 2, D, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    q = q.to(dev)
    table = torch.arange(pages, dtype=torch.int32, device=dev).view(1, -1)
    scale = 0.6931471805599453  # of q . k in powers of two
    # the weights' bf16 rounding, the output's, and the sums' (exponents of weights are off by 2^-18 at most)
    near = lambda got: ((got.cpu().double() / 2.0 ** exponent - 1).abs() <=
                        2 * ref.EPS16 + 2 * (length + 40) * ref.EPS32 + steps_below(length, 8) / 2.0 ** exponent + 2.0 ** -18).all()
    assert near(ql.attn_decode(q[:1], cache, table, ints([length], dev), scale=scale))
    n = min(3, length)
    assert near(ql.attn_prompt(q[:n], ints([0, n], dev), cache, table, ints([length], dev), scale=scale))


@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
def test_one_token_of_any_stride(dev, ty):
    Hq, Hkv, D = 4, 2, 64
    rows = [torch.randn(1, h * D, generator=torch.Generator().manual_seed(h)).to(ty).to(dev) for h in (Hq, Hkv, Hkv)]
    odd = [torch.empty(x.shape[1], 1, dtype=ty, device=dev).t().copy_(x) for x in rows]
    assert all(x.is_contiguous() and x.stride() == (1, 1) for x in odd)
    rope = ql.Rope(torch.rand(D // 2, device=dev))
    results = []
    for q, k, v in (rows, odd):
        cache = ql.KvCache(*(torch.zeros(1, Hkv, 16, D, dtype=torch.bfloat16, device=dev) for _ in "kv"))
        turned = ql.rope_append(q, k, v, ints([7], dev), ints([3], dev), rope, cache)
        y = ql.attn_decode(turned, cache, ints([[0]], dev), ints([4], dev))
        z = ql.attn_prompt(turned.t().contiguous().t(), ints([0, 1], dev), cache, ints([[0]], dev), ints([4], dev))
        results.append((turned, cache.k, cache.v, y, z))
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("spread,eps", [(1e30, 1e-6), (1e37, 0.0), (1e19, 1e-6), (1e18, 1e38), (1e-12, 0.0), (1e-18, 1e-36), (1e-22, 0.0),
                                        (1e-30, 1e-38), (1e-36, 0.0)])
@pytest.mark.parametrize("D", [64, 128])
def test_norms_of_any_size(dev, ty, spread, eps, D):
    """Squares that fp32 does not hold: the norm is what it is for any other size."""
    T, H = 5, 3
    g = torch.Generator().manual_seed(D)
    x = (torch.randn(T, H, D, generator=g) * spread).to(ty)
    x[:, 1] *= 2.0 ** -10  # heads of another size beside
    norm = 1 + 0.2 * torch.randn(D, generator=g)
    positions = torch.arange(T, dtype=torch.int32)
    freqs = torch.rand(D // 2, generator=g)
    cache = ql.KvCache(*(torch.zeros(1, H, 16, D, dtype=torch.bfloat16, device=dev) for _ in "kv"))
    got = ql.rope_append(*(x.to(dev),) * 3, positions.to(dev), positions.to(dev), ql.Rope(freqs.to(dev)), cache, q_norm=norm.to(dev),
                         k_norm=norm.to(dev), eps=eps)
    want, slack = ref.turned(x, positions, freqs, False, 1.0, norm, torch.tensor(eps, dtype=torch.float32).double())
    # (an eps of fewer bits, fp32's last step beside it)
    slack = slack + (2.0 ** -150 / eps if eps else 0.0) * want.abs()
    assert ref.bf16_close(got.cpu(), want, slack).all()
    assert ref.bf16_close(cache.k.cpu()[0, :, :T].transpose(0, 1), want, slack).all()


@pytest.mark.parametrize("starts,ranges", [([-3, 20, 10, 10], [(0, 20), (20, 20), (10, 10)]), ([0, 25, 10 ** 9], [(0, 25), (25, 40)]),
                                           ([-(2 ** 31), -1, 7, 2 ** 31 - 1], [(0, 0), (0, 7), (7, 40)]), ([50, 60, 10 ** 9], [(40, 40)] * 2)])
@pytest.mark.parametrize("length", [40, 3000])
def test_rows_of_cut_starts(dev, starts, ranges, length):
    """starts are cut to 0 .. T, a range that ends before it begins is empty; the rows left have their results, no other row
    is written, and none around q is read into them."""
    T, Hq, D = 40, 2, 64
    seqs = ref.Sequences([length] * len(ranges), 1, D, 16, seed=8)
    cache, table, lens = seqs.on(dev)
    room = 200 * Hq * D
    held = torch.full((T * Hq * D + 2 * room,), float("nan"), dtype=torch.bfloat16, device=dev)
    out = torch.full_like(held, 5.0)
    q, y = (t[room:-room].view(T, Hq, D) for t in (held, out))
    q.copy_(ref.queries(T, Hq, D, 9))
    ql.attn_prompt(q, ints(starts, dev), cache, table, lens, out=y)
    assert (out[:room] == 5.0).all() and (out[-room:] == 5.0).all()
    mine = torch.zeros(T, dtype=torch.bool)
    y, host = y.cpu(), q.cpu()
    for b, (first, end) in enumerate(ranges):
        if first == end:
            continue
        mine[first:end] = True
        k, v = seqs.kv[b]
        sees = torch.arange(length)[None] <= length - (end - first) + torch.arange(end - first)[:, None]
        want, slack = ref.attention(host[first:end], k, v, sees, D ** -0.5)
        assert ref.bf16_close(y[first:end], want, slack).all()
    assert (y[~mine] == 5.0).all()


def test_scores_of_minus_infinity(dev):
    """Such a key weighs 0, and a row of no other keys is 0."""
    D, n = 64, 40
    seqs = ref.Sequences([n, 5], 1, D, 16, seed=2)
    q = ref.queries(2, 2, D, 3).abs() + 1
    visible = torch.ones(n, dtype=torch.bool)
    for i in (3, 17, 39):
        seqs.k[seqs.table[0, i // 16], 0, i % 16, 5] = -float("inf")
        visible[i] = False
    seqs.k[seqs.table[1, 0], 0, :5, 7] = -float("inf")
    cache, table, lens = seqs.on(dev)
    want, slack = ref.decode(seqs, q, D ** -0.5, {0: visible})
    for got in (ql.attn_decode(q.to(dev), cache, table, lens), ql.attn_prompt(q.to(dev), ints([0, 1, 2], dev), cache, table, lens)):
        assert ref.bf16_close(got.cpu()[:1], want[:1], slack[:1]).all() and (got[1] == 0).all()
