"""Attention of one new token and of packed prompts over the paged cache, on the GPU against a plain 64-bit
reference, and a whole step (products, rotary positions, cache, attention, product) eager and in a graph."""
import numpy as np
import pytest
import torch

import attn_reference as ref
from decode_gemv_thinkbit_amd import qlinear as ql

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 300]


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ql.lib()
    return torch.device("cuda:0")


def close(got, want, slack):
    ok = ref.bf16_close(got.cpu().view(want.shape), want, slack)
    assert ok.all(), (int((~ok).sum()), ok.numel(), ((got.cpu().view(want.shape).double() - want).abs() - slack).max())


# ---------------------------------------------------------------- one new token
def check_decode(dev, lens, Hq, Hkv, D, page, cache="bf16", seed=0, spread=1.0, scale=None, **more):
    seqs = ref.Sequences(lens, Hkv, D, page, cache, seed, **more)
    q = ref.queries(len(lens), Hq, D, seed + 1, spread)
    got = ql.attn_decode(q.to(dev), *seqs.on(dev), scale=scale)
    assert got.dtype == torch.bfloat16 and got.shape == q.shape
    want, slack = ref.decode(seqs, q, D ** -0.5 if scale is None else scale)
    close(got, want, slack)
    for b, n in enumerate(lens):
        if n <= 0:
            assert (got[b] == 0).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
def test_decode_lengths(dev, cache, D, page):
    check_decode(dev, EDGES, 4, 2, D, page, cache, seed=page)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_lengths_in_chunks(dev, cache, D):
    """The same where one sequence is long enough for all to go by chunks."""
    check_decode(dev, EDGES + [511, 512, 513, 640, 641], 4, 2, D, 16, cache, seed=D)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (5, 1), (14, 2), (16, 1), (17, 1), (40, 2), (32, 1), (64, 8)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_decode_heads(dev, Hq, Hkv, cache):
    check_decode(dev, [70, 1, 0, 700], Hq, Hkv, 128, 32, cache, seed=Hq)
    check_decode(dev, [515], Hq, Hkv, 64, 16, cache, seed=Hq + 1)


@pytest.mark.parametrize("lens", [[9000], [20011, 3, 0, 513], [1] * 130, [(37 * b) % 1500 for b in range(200)], [65536],
                                  [(13 * b) % 700 for b in range(600)], [257] * 256, [1] * 257 + [3000]])
@pytest.mark.parametrize("D,cache", [(128, "bf16"), (64, "e4m3")])
def test_decode_split_and_batches(dev, lens, D, cache):
    check_decode(dev, lens, 4, 1, D, 16, cache, seed=len(lens))


@pytest.mark.parametrize("spread,scale", [(8.0, None), (30.0, 1.0), (0.0, None), (1.0, 1e-6), (1e-20, 1.0)])
def test_decode_score_ranges(dev, spread, scale):
    check_decode(dev, [300, 33, 1000], 4, 2, 128, 16, seed=7, spread=spread, scale=scale)


def test_decode_garbage_behind_the_end(dev):
    """What unused slots and pages hold does not matter, NaN and infinities neither."""
    for cache, fill in (("bf16", NAN), ("bf16", INF), ("e4m3", NAN)):
        check_decode(dev, EDGES, 4, 2, 128, 64, cache, seed=11, fill=fill)


def test_decode_bad_pages(dev):
    """Entries that are no page: their tokens are not seen."""
    seqs = ref.Sequences([200, 64, 16, 3000], 2, 128, 16, seed=5, fill=NAN, spare=0)
    q = ref.queries(4, 4, 128, 6)
    cache, table, lens = seqs.on(dev)
    visible = {}
    for b, entries in ((0, {0: -1, 5: 10 ** 9}), (1, {1: -5, 2: seqs.k.shape[0], 3: 2 ** 31 - 1}), (2, {0: -2 ** 31}),
                       (3, {i: -1 for i in range(60, 120)})):
        visible[b] = torch.ones(seqs.lens[b], dtype=torch.bool)
        for i, e in entries.items():
            table[b, i] = e
            visible[b][16 * i : 16 * i + 16] = False
    cache.k[seqs.table[0, 0].item()] = NAN  # a page that is seen by nobody now
    cache.v[seqs.table[0, 0].item()] = NAN
    got = ql.attn_decode(q.to(dev), cache, table, lens)
    want, slack = ref.decode(seqs, q, 128 ** -0.5, visible)
    close(got, want, slack)
    assert (got[2] == 0).all()


def test_decode_lengths_outside(dev):
    """Lengths below 0 are none, those past the table's row are cut to it."""
    seqs = ref.Sequences([48, 48, 48], 1, 64, 16, seed=8)
    q = ref.queries(3, 2, 64, 9)
    cache, table, _ = seqs.on(dev)
    want = ql.attn_decode(q.to(dev), cache, table, torch.tensor([0, 48, 48], dtype=torch.int32, device=dev))
    got = ql.attn_decode(q.to(dev), cache, table, torch.tensor([-9, 49, 2 ** 31 - 1], dtype=torch.int32, device=dev))
    assert torch.equal(got, want) and (got[0] == 0).all()


def test_decode_infinite_values(dev):
    """A visible infinity of V comes out, of its own dim alone; a NaN key's sequence is NaN."""
    seqs = ref.Sequences([40, 300], 1, 64, 16, seed=3)
    q = ref.queries(2, 2, 64, 4)
    cache, table, lens = seqs.on(dev)
    want = ql.attn_decode(q.to(dev), cache, table, lens)
    cache.v[seqs.table[0, 1].item(), 0, 5, 7] = INF
    cache.k[seqs.table[1, 3].item(), 0, 2, 9] = NAN
    got = ql.attn_decode(q.to(dev), cache, table, lens)
    assert (got[0, :, 7] == INF).all() and torch.isnan(got[1]).all()
    keep = [d for d in range(64) if d != 7]
    assert torch.equal(got[0][:, keep], want[0][:, keep])


def of_large_values(seqs):
    """V as large as its type allows: sums of a few would pass fp32's end."""
    most = 2.0 ** 125
    seqs.v = seqs.v.abs() * most
    for both in seqs.kv:
        both[1] = both[1].abs() * most
    return seqs


@pytest.mark.parametrize("lens", [[500], [700, 3, 40], [9000]])
def test_decode_large_values(dev, lens):
    seqs = of_large_values(ref.Sequences(lens, 2, 64, 16, seed=5))
    q = ref.queries(len(lens), 4, 64, 6)
    want, slack = ref.decode(seqs, q, 64 ** -0.5)
    close(ql.attn_decode(q.to(dev), *seqs.on(dev)), want, slack)


@pytest.mark.parametrize("n,length", [(200, 200), (300, 300), (700, 700), (5, 4000), (300, 4000)])
def test_prompt_large_values(dev, n, length):
    seqs = of_large_values(ref.Sequences([length], 2, 128, 16, seed=5))
    q = ref.queries(n, 4, 128, 6)
    cache, table, lens = seqs.on(dev)
    got = ql.attn_prompt(q.to(dev), torch.tensor([0, n], dtype=torch.int32, device=dev), cache, table, lens)
    want, slack = ref.prompt(seqs, q, [0, n], 128 ** -0.5)
    close(got, want, slack)


def test_decode_equal_scores_average(dev):
    """Equal keys: the mean of V."""
    n = 777
    k = torch.ones(64, 1, 16, 64, dtype=torch.bfloat16, device=dev)
    v = torch.arange(64 * 16, device=dev).remainder(7).to(torch.bfloat16).view(64, 1, 16, 1).expand(64, 1, 16, 64).contiguous()
    table = torch.arange(64, dtype=torch.int32, device=dev).view(1, 64)
    got = ql.attn_decode(torch.ones(1, 3, 64, dtype=torch.bfloat16, device=dev), ql.KvCache(k, v), table,
                         torch.tensor([n], dtype=torch.int32, device=dev))
    want = torch.tensor(np.mean(np.arange(n) % 7))
    assert ((got.cpu().double() - want).abs() <= want * ref.EPS16 * 2).all()


# ---------------------------------------------------------------- packed prompts
def check_prompt(dev, new, before, Hq, Hkv, D, page, cache="bf16", seed=0, spread=1.0, behind=0, visible=None, **more):
    lens = [n + p for n, p in zip(new, before)]
    seqs = ref.Sequences(lens, Hkv, D, page, cache, seed, **more)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    T = max(1, starts[-1] + behind)
    q = ref.queries(T, Hq, D, seed + 1, spread)
    c, table, ln = seqs.on(dev)
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=dev)
    got = ql.attn_prompt(q.to(dev), torch.tensor(starts, dtype=torch.int32, device=dev), c, table, ln, out=out)
    assert got is out
    want, slack = ref.prompt(seqs, q, starts, D ** -0.5)
    close(got[: starts[-1]], want[: starts[-1]], slack[: starts[-1]])
    assert (got[starts[-1] :] == 5.0).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_prompt_lengths(dev, cache, D, page):
    new = [n for n in EDGES if n < 140]
    check_prompt(dev, new, [0] * len(new), 4, 2, D, page, cache, seed=page, behind=9)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (5, 1), (14, 2), (8, 1), (20, 1), (130, 1)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_prompt_heads(dev, Hq, Hkv, cache):
    check_prompt(dev, [70, 1, 0, 33], [0, 5, 9, 200], Hq, Hkv, 128, 32, cache, seed=Hq)
    check_prompt(dev, [65], [0], Hq, Hkv, 64, 16, cache, seed=Hq + 1)


@pytest.mark.parametrize("new,before", [([600], [0]), ([1], [4000]), ([5, 1, 17], [3000, 0, 700]), ([257], [2000]),
                                        ([1] * 70, [(61 * b) % 900 for b in range(70)]), ([300, 900, 10], [0, 0, 0])])
@pytest.mark.parametrize("D,cache", [(128, "bf16"), (64, "bf16"), (128, "e4m3")])
def test_prompt_chunks_and_splits(dev, new, before, D, cache):
    check_prompt(dev, new, before, 4, 2, D, 16, cache, seed=len(new) + D)


@pytest.mark.parametrize("B", [64, 65, 140])
def test_prompt_many_sequences(dev, B):
    """Of every length, equal ones and empty ones among them: their tiles' order is not the batch's."""
    check_prompt(dev, [(7 * b) % 40 for b in range(B)], [(37 * b) % 300 if b % 3 else 0 for b in range(B)], 8, 1, 64, 16, seed=B)


@pytest.mark.parametrize("new,before,Hq,Hkv", [([2500], [0], 16, 16), ([4200], [0], 16, 16), ([1500, 9, 1100], [0, 0, 0], 16, 8),
                                               ([500], [5000], 16, 4), ([400, 130], [4000, 6000], 8, 4), ([1300], [0], 16, 16),
                                               ([1700], [0], 24, 8)])
def test_prompt_more_tiles_than_first_workgroups(dev, new, before, Hq, Hkv):
    """More row tiles than the CUs take at first: the others' order differs, in parts of rows too."""
    check_prompt(dev, new, before, Hq, Hkv, 64, 64, seed=len(new))


def test_prompt_rows_that_see_nothing(dev):
    """More queries than tokens: the first see nothing."""
    check_prompt(dev, [20, 200, 3], [-15, -200, -1], 4, 2, 128, 16, seed=4)


@pytest.mark.parametrize("spread", [8.0, 30.0, 0.0])
def test_prompt_score_ranges(dev, spread):
    check_prompt(dev, [200, 33], [0, 100], 4, 2, 128, 16, seed=7, spread=spread)


def test_prompt_rows_in_front_of_the_first_sequence(dev):
    """Rows before starts[0], as those behind the last sequence, are left as they were."""
    seqs = ref.Sequences([40, 9], 1, 64, 16, seed=8)
    q = ref.queries(60, 2, 64, 9)
    cache, table, lens = seqs.on(dev)
    starts = [5, 45, 54]
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=dev)
    ql.attn_prompt(q.to(dev), torch.tensor(starts, dtype=torch.int32, device=dev), cache, table, lens, out=out)
    want, slack = ref.prompt(seqs, q, starts, 64 ** -0.5)
    close(out[5:54], want[5:54], slack[5:54])
    assert (out[:5] == 5.0).all() and (out[54:] == 5.0).all()


def test_prompt_garbage_behind_the_end(dev):
    new = [n for n in EDGES if n < 140]
    for cache, fill in (("bf16", NAN), ("bf16", -INF), ("e4m3", NAN)):
        check_prompt(dev, new, [0] * len(new), 4, 2, 128, 64, cache, seed=11, fill=fill)


def test_prompt_infinite_values_stay_with_the_rows_that_see_them(dev):
    for D, G, before in ((128, 2, 0), (64, 3, 0), (128, 1, 3000)):
        n = 150
        seqs = ref.Sequences([before + n], 1, D, 16, seed=3)
        q = ref.queries(n, G, D, 4)
        cache, table, lens = seqs.on(dev)
        starts = torch.tensor([0, n], dtype=torch.int32, device=dev)
        want = ql.attn_prompt(q.to(dev), starts, cache, table, lens)

        def put(t, at, d, x):
            t[seqs.table[0, (before + at) // 16].item(), 0, (before + at) % 16, d] = x

        put(cache.v, 100, 7, INF)
        put(cache.v, 60, 33, -INF)
        put(cache.v, 129, 33, INF)  # meets the one above
        put(cache.v, 20, 50, NAN)
        got = ql.attn_prompt(q.to(dev), starts, cache, table, lens)
        change = {7: [(100, INF)], 33: [(60, -INF), (129, NAN)], 50: [(20, NAN)]}
        expect = want.clone()
        for d, at in change.items():
            for first, x in at:
                expect[first:, :, d] = x
        assert torch.equal(torch.isnan(got), torch.isnan(expect))
        assert torch.equal(torch.nan_to_num(got, nan=3.0), torch.nan_to_num(expect, nan=3.0))
        put(cache.k, 90, 1, NAN)
        got = ql.attn_prompt(q.to(dev), starts, cache, table, lens)
        assert torch.isnan(got[90:]).all()
        assert torch.equal(torch.nan_to_num(got[:90], nan=3.0), torch.nan_to_num(expect[:90], nan=3.0))


def test_prompt_bad_pages(dev):
    seqs = ref.Sequences([200, 1700], 2, 128, 16, seed=5, fill=NAN, spare=0)
    starts = [0, 150, 190]
    q = ref.queries(190, 4, 128, 6)
    cache, table, lens = seqs.on(dev)
    visible = {}
    for b, entries in ((0, {0: -1, 5: 10 ** 9, 12: seqs.k.shape[0]}), (1, {i: -1 for i in range(20, 90)})):
        visible[b] = torch.ones(seqs.lens[b], dtype=torch.bool)
        for i, e in entries.items():
            table[b, i] = e
            visible[b][16 * i : 16 * i + 16] = False
    cache.v[seqs.table[0, 0].item()] = NAN
    cache.k[seqs.table[0, 0].item()] = NAN
    got = ql.attn_prompt(q.to(dev), torch.tensor(starts, dtype=torch.int32, device=dev), cache, table, lens)
    want, slack = ref.prompt(seqs, q, starts, 128 ** -0.5, visible)
    close(got, want, slack)


@pytest.mark.parametrize("D,G,cache", [(128, 2, "bf16"), (64, 3, "bf16"), (128, 1, "e4m3")])
def test_prompt_long_rows_infinities_and_bad_pages(dev, D, G, cache):
    """Rows long enough for two groups of waves, of which each has every second tile of 64 keys."""
    n = 450
    seqs = ref.Sequences([n], 1, D, 16, cache, seed=3)
    q = ref.queries(n, G, D, 4)
    kv, table, lens = seqs.on(dev)
    starts = torch.tensor([0, n], dtype=torch.int32, device=dev)
    call = lambda: ql.attn_prompt(q.to(dev), starts, kv, table, lens)
    visible = torch.ones(n, dtype=torch.bool)
    for i, e in {1: -1, 5: 10 ** 9, 14: -7, 23: seqs.k.shape[0]}.items():
        table[0, i] = e
        visible[16 * i : 16 * i + 16] = False
    want = call()
    exact, slack = ref.prompt(seqs, q, [0, n], D ** -0.5, {0: visible})
    close(want, exact, slack)

    def put(t, at, d, x):
        t.view(torch.uint8 if cache == "e4m3" else t.dtype)[seqs.table[0, at // 16].item(), 0, at % 16, d] = x

    nan = 0x7F if cache == "e4m3" else NAN
    expect = want.clone()
    for at, d in ((50, 7), (100, 9), (330, 3), (449, 60)):
        put(kv.v, at, d, nan)
        expect[at:, :, d] = NAN
    if cache == "bf16":
        for at, d, x in ((70, 33, INF), (140, 33, -INF), (200, 40, -INF), (270, 40, -INF)):
            put(kv.v, at, d, x)
            expect[at:, :, d] = NAN if at == 140 else x
    put(kv.v, 20, 11, nan)  # of a page that is not seen
    got = call()
    assert torch.equal(torch.isnan(got), torch.isnan(expect))
    assert torch.equal(torch.nan_to_num(got, nan=3.0), torch.nan_to_num(expect, nan=3.0))


def test_prompt_starts_are_cut(dev):
    """starts outside 0 .. T are cut to it and a range that ends before it begins is empty: nothing else is read or written."""
    seqs = ref.Sequences([40, 40, 40], 1, 64, 16, seed=8)
    q = ref.queries(40, 2, 64, 9)
    cache, table, lens = seqs.on(dev)
    out = torch.full_like(q, 5.0, device=dev)
    ql.attn_prompt(q.to(dev), torch.tensor([-3, 40, 20, 10 ** 9], dtype=torch.int32, device=dev)[:4], cache, table, lens, out=out)
    assert torch.isfinite(out).all()


def test_prompt_of_single_tokens_is_decode(dev):
    lens = [1, 50, 700, 2000]
    seqs = ref.Sequences(lens, 2, 128, 16, seed=21)
    q = ref.queries(4, 8, 128, 22)
    cache, table, ln = seqs.on(dev)
    got = ql.attn_prompt(q.to(dev), torch.arange(5, dtype=torch.int32, device=dev), cache, table, ln)
    want, slack = ref.decode(seqs, q, 128 ** -0.5)
    close(got, want, slack)


# ---------------------------------------------------------------- how they are called
def test_memory_around_strides_and_determinism(dev):
    """Results go to `out` alone; a table's rows may be part of wider ones; the same call gives the same bits."""
    lens = [5000, 3, 0, 900]
    seqs = ref.Sequences(lens, 2, 128, 16, seed=31)
    cache, table, ln = seqs.on(dev)
    wide = torch.full((4, seqs.most + 50), 10 ** 9, dtype=torch.int32, device=dev)
    wide[:, 3 : 3 + seqs.most] = table
    q = ref.queries(4, 8, 128, 32).to(dev)
    for call in (lambda t, **kw: ql.attn_decode(q, cache, t, ln, **kw),
                 lambda t, **kw: ql.attn_prompt(q, torch.arange(5, dtype=torch.int32, device=dev), cache, t, ln, **kw)):
        want = call(table)
        buf = torch.full((q.numel() + 256,), -3.0, dtype=torch.bfloat16, device=dev)
        out = buf[128:-128].view(q.shape)
        assert call(wide[:, 3 : 3 + seqs.most], out=out) is out
        assert torch.equal(out, want) and (buf[:128] == -3).all() and (buf[-128:] == -3).all()
        assert torch.equal(call(table), want)
    flat = ql.attn_decode(q.view(4, -1), cache, table, ln)
    assert flat.shape == (4, 1024) and torch.equal(flat.view(q.shape), ql.attn_decode(q, cache, table, ln))


def test_offsets_beyond_32_bits(dev):
    """Pages past 4 GiB of the cache."""
    pages, Hkv, page, D = 2100, 8, 1024, 128
    k, v = (torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device=dev) for _ in "kv")
    assert 2 * pages * Hkv * page * D > 1 << 32
    seqs = ref.Sequences([2100], Hkv, D, page, seed=41, spare=0)
    ids = [pages - 1, 0, pages - 2]
    for i, p in enumerate(ids):
        k[p], v[p] = (t[seqs.table[0, i].item()].to(dev) for t in (seqs.k, seqs.v))
    table = torch.tensor([ids], dtype=torch.int32, device=dev)
    ln = torch.tensor([2100], dtype=torch.int32, device=dev)
    q = ref.queries(40, 8, D, 42)
    got = ql.attn_decode(q[39:].to(dev), ql.KvCache(k, v), table, ln)
    close(got, *ref.decode(seqs, q[39:], D ** -0.5))
    got = ql.attn_prompt(q.to(dev), torch.tensor([0, 40], dtype=torch.int32, device=dev), ql.KvCache(k, v), table, ln)
    close(got, *ref.prompt(seqs, q, [0, 40], D ** -0.5))


def test_two_streams(dev):
    """Two calls at once, each on a stream and with a workspace of its own."""
    seqs = ref.Sequences([6000, 700], 2, 128, 16, seed=51)
    cache, table, ln = seqs.on(dev)
    qs = [ref.queries(2, 8, 128, 52 + i).to(dev) for i in range(2)]
    want = [ql.attn_decode(q, cache, table, ln) for q in qs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in qs], [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ql.attn_decode(qs[i], cache, table, ln))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


class Layer:
    """What a decode step does between a layer's input and its attention's output: q, k, v products of low-bit
    weights in one grouped launch, rotary positions and cache, attention, the output product."""

    def __init__(self, dev, B, Hq=8, Hkv=2, D=128, hidden=640, page=16, most=8):
        g = torch.Generator().manual_seed(61)
        self.B, self.Hq, self.Hkv, self.D, self.hidden = B, Hq, Hkv, D, hidden
        weight = lambda n, k: ql.quantize_pack((torch.randn(n, k, generator=g) * 0.05).to(dev), ql.GRID_I3)
        self.w = [weight(n * D, hidden) for n in (Hq, Hkv, Hkv)]
        self.wo = weight(hidden, Hq * D)
        self.x = torch.zeros(B, hidden, dtype=torch.bfloat16, device=dev)
        self.y = [torch.empty(B, n * D, device=dev) for n in (Hq, Hkv, Hkv)]
        self.qkv = ql.GroupedGemv([(w, self.x, y) for w, y in zip(self.w, self.y)])
        self.cache = ql.KvCache(*(torch.zeros(B * most, Hkv, page, D, dtype=torch.bfloat16, device=dev) for _ in "kv"))
        self.table = torch.randperm(B * most, generator=g).int().view(B, most).to(dev)
        self.rope = ql.Rope(ql.rope_frequencies(D, 1e6)[0].to(dev))
        self.norms = [(1 + 0.1 * torch.randn(D, generator=g)).to(dev) for _ in "qk"]
        self.positions, self.slots, self.lens = (torch.zeros(B, dtype=torch.int32, device=dev) for _ in range(3))
        self.q = torch.empty(B, Hq * D, dtype=torch.bfloat16, device=dev)
        self.attn = torch.empty_like(self.q)
        self.out = torch.empty(B, hidden, device=dev)
        need = ql.lib().qlinear_attn_decode_workspace_bytes(B, Hq, Hkv, D, most * page)
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)

    def set_step(self, x, lens):
        """x [B, hidden], the tokens in front of this one."""
        self.x.copy_(x)
        self.positions.copy_(lens)
        page = self.cache.shape[2]
        self.slots.copy_(self.table.gather(1, (lens // page).long()[:, None])[:, 0] * page + lens % page)
        self.lens.copy_(lens + 1)

    def run(self):
        self.qkv.run()
        ql.rope_append(*self.y, self.positions, self.slots, self.rope, self.cache, q_norm=self.norms[0],
                       k_norm=self.norms[1], out=self.q)
        ql.attn_decode(self.q, self.cache, self.table, self.lens, out=self.attn, workspace=self.ws)
        ql.gemv(self.attn, self.wo, out=self.out)
        return self.out


def test_a_layer_step_by_step_eager_and_in_a_graph(dev):
    """Decoding tokens one by one gives what the prompt's attention gives for all of them at once, and a captured
    step replays with new inputs, eager work between the replays."""
    B, steps = 3, 40
    layer = Layer(dev, B)
    g = torch.Generator().manual_seed(62)
    xs = torch.randn(steps, B, layer.hidden, generator=g).to(torch.bfloat16).to(dev)
    eager = []
    for i in range(steps):
        layer.set_step(xs[i], torch.full((B,), i, dtype=torch.int32, device=dev))
        eager.append((layer.run().clone(), layer.q.clone(), layer.attn.clone()))
    # all at once: the queries of every step against the cache that they left
    q = torch.stack([e[1] for e in eager], 1).view(B * steps, -1)
    starts = torch.arange(B + 1, dtype=torch.int32, device=dev) * steps
    whole = ql.attn_prompt(q, starts, layer.cache, layer.table, torch.full((B,), steps, dtype=torch.int32, device=dev))
    whole = whole.view(B, steps, -1)
    held = [t.float().cpu() for t in (layer.cache.k, layer.cache.v)]
    page = layer.cache.shape[2]
    seqs = ref.Sequences([0] * B, layer.Hkv, layer.D, page)
    for b in range(B):
        rows = layer.table[b].cpu().long()
        seqs.kv[b] = [t[rows].transpose(1, 2).reshape(-1, layer.Hkv, layer.D)[:steps].double() for t in held]
    want, slack = ref.prompt(seqs, q.cpu().view(-1, layer.Hq, layer.D), starts.tolist(), layer.D ** -0.5)
    close(whole.reshape(-1, layer.Hq * layer.D), want, slack)
    close(torch.stack([e[2] for e in eager], 1).reshape(-1, layer.Hq * layer.D), want, slack)
    # captured
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        layer.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run()
    layer.cache.k.zero_()
    layer.cache.v.zero_()
    for i in range(steps):
        layer.set_step(xs[i], torch.full((B,), i, dtype=torch.int32, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out, eager[i][0]) and torch.equal(layer.attn, eager[i][2])
        torch.randn(1000, device=dev).sum()  # eager work between the replays


def test_prompt_then_decode(dev):
    """A packed prompt through the products of the GEMM, then one more token: what the 64-bit reference gives."""
    dev_t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    Hq, Hkv, D, page, hidden = 4, 2, 64, 16, 256
    new = [37, 50, 16]
    T = sum(new)
    g = torch.Generator().manual_seed(71)
    w = ql.quantize_pack((torch.randn((Hq + 2 * Hkv) * D, hidden, generator=g) * 0.1).to(dev), ql.GRID_I2)
    x = torch.randn(T, hidden, generator=g).to(torch.bfloat16).to(dev)
    cache = ql.KvCache(*(torch.zeros(20, Hkv, page, D, dtype=torch.bfloat16, device=dev) for _ in "kv"))
    table = torch.randperm(20, generator=g)[:15].int().view(3, 5)
    rope = ql.Rope(ql.rope_frequencies(D)[0].to(dev), interleaved=True)
    where = [(b, i) for b, n in enumerate(new) for i in range(n)]
    slot = lambda b, i: int(table[b, i // page]) * page + i % page
    rows = ql.gemm(x, w).split((Hq * D, Hkv * D, Hkv * D), 1)  # one fused product, parts of its rows
    q = ql.rope_append(*rows, dev_t([i for _, i in where]), dev_t([slot(b, i) for b, i in where]), rope, cache)
    out = ql.attn_prompt(q, dev_t([0, 37, 87, 103]), cache, table.to(dev), dev_t(new))
    x1 = torch.randn(3, hidden, generator=g).to(torch.bfloat16).to(dev)
    rows = ql.gemv(x1, w).split((Hq * D, Hkv * D, Hkv * D), 1)
    q1 = ql.rope_append(*rows, dev_t(new), dev_t([slot(b, n) for b, n in enumerate(new)]), rope, cache)
    out1 = ql.attn_decode(q1, cache, table.to(dev), dev_t([n + 1 for n in new]))
    seqs = ref.Sequences([0] * 3, Hkv, D, page)
    full = []
    for b, n in enumerate(new):
        full.append([t.cpu()[table[b].long()].transpose(1, 2).reshape(-1, Hkv, D).double() for t in (cache.k, cache.v)])
        seqs.kv[b] = [t[:n] for t in full[b]]
    close(out, *ref.prompt(seqs, q.cpu().view(T, Hq, D), [0, 37, 87, 103], D ** -0.5))
    for b, n in enumerate(new):
        seqs.kv[b] = [t[: n + 1] for t in full[b]]
    close(out1, *ref.decode(seqs, q1.cpu().view(3, Hq, D), D ** -0.5))


@pytest.mark.parametrize("B,capacity", [(1, 1280), (3, 1280), (1, 4096), (2, 4096)])
def test_prompt_chunks_replayed(dev, B, capacity):
    """Chunks of packed prompts through rope_append and attn_prompt in one captured graph: other lengths, positions and
    values each time, eager work between, the bits of eager calls on a cache of their own."""
    T, Hq, Hkv, D, page = 320, 4, 2, 64, 16
    g = torch.Generator().manual_seed(71)
    pages = B * capacity // page
    table = torch.randperm(pages, generator=g).int().view(B, -1)
    caches = [ql.KvCache(*(torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device=dev) for _ in "kv")) for _ in "ab"]
    rope = ql.Rope(ql.rope_frequencies(D)[0].to(dev))
    q, k, v = (torch.zeros(T, h, D, device=dev) for h in (Hq, Hkv, Hkv))
    positions, slots = (torch.full((T,), -1, dtype=torch.int32, device=dev) for _ in "ps")
    starts, lens = torch.zeros(B + 1, dtype=torch.int32, device=dev), torch.zeros(B, dtype=torch.int32, device=dev)
    at, out = table.to(dev), torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)

    def step(cache):
        return ql.attn_prompt(ql.rope_append(q, k, v, positions, slots, rope, cache), starts, cache, at, lens, out=out)

    done = [0] * B

    def fill(i):
        cuts = sorted(torch.randint(0, T - 9, (B - 1,), generator=g).tolist())
        new = [b - a for a, b in zip([0] + cuts, cuts + [T - 5 * i])]  # the last rows are nobody's
        p, s, begin = [], [], [0]
        for b in range(B):
            where = torch.arange(done[b], done[b] + new[b])
            p.append(where)
            s.append(table[b, where // page] * page + where % page)
            done[b] += new[b]
            begin.append(begin[-1] + new[b])
        rest = T - begin[-1]
        positions.copy_(torch.cat(p + [torch.zeros(rest)]).int())
        slots.copy_(torch.cat(s + [torch.full((rest,), -1)]).int())
        starts.copy_(torch.tensor(begin).int())
        lens.copy_(torch.tensor(done).int())
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):  # no token has a slot, no sequence a row
        step(caches[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[1])
    for c in caches:
        c.k.zero_(), c.v.zero_()
    for i in range(3):
        fill(i)
        out.fill_(5.0)
        want = step(caches[0]).clone()
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
        torch.randn(1000, device=dev).sum()
    n = starts.tolist()
    turned = ql.rope_append(q, k, v, positions, slots, rope, caches[0]).cpu()
    seqs = ref.Sequences([0] * B, Hkv, D, page)
    for b in range(B):
        seqs.kv[b] = [t.float().cpu()[table[b].long()].transpose(1, 2).reshape(-1, Hkv, D)[: done[b]].double()
                      for t in (caches[0].k, caches[0].v)]
    want, slack = ref.prompt(seqs, turned, n, D ** -0.5)
    close(out[: n[-1]], want[: n[-1]], slack[: n[-1]])
    assert (out[n[-1] :] == 5.0).all()
