"""Rotary positions and the paged cache's filling on the GPU against a plain 64-bit reference."""
import math

import pytest
import torch

import attn_reference as ref
from decode_gemv_thinkbit_amd import qlinear as ql

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ql.lib()
    return torch.device("cuda:0")


def empty_cache(pages, Hkv, page, D, kind, dev, fill=0.0):
    store = [torch.full((pages, Hkv, page, D), fill).to(ref.F8 if kind == "e4m3" else torch.bfloat16).to(dev) for _ in "kv"]
    scales = [torch.linspace(0.5, 2.0, Hkv).to(dev) * s for s in (0.01, 0.02)] if kind == "e4m3" else [None, None]
    return ql.KvCache(*store, *scales)


def check(dev, T, Hq, Hkv, D, R, ty=torch.float32, kind="bf16", page=16, inter=False, norm=False, factor=1.0, far=5000,
          fused=True, seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    widths = (Hq * D, Hkv * D, Hkv * D)
    rows = (torch.randn(T, sum(widths), generator=g) * spread).to(ty)
    q, k, v = rows.split(widths, 1)
    q, k, v = (x.unflatten(1, (-1, D)) for x in (q, k, v))
    positions = torch.randint(0, far, (T,), generator=g).int()
    pages = (T + page - 1) // page + 2
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    slots[torch.rand(T, generator=g) < 0.1] = -1
    freqs = (1e6 ** (-torch.arange(0, R, 2).double() / R)).float()
    norms = [(1 + 0.2 * torch.randn(D, generator=g)) for _ in "qk"] if norm else [None, None]
    cache = empty_cache(pages, Hkv, page, D, kind, dev)
    on = rows.to(dev)
    parts = on.split(widths, 1) if fused else [x.reshape(T, -1, D).contiguous().to(dev) for x in (q, k, v)]
    got = ql.rope_append(*parts, positions.to(dev), slots.to(dev), ql.Rope(freqs.to(dev), inter, factor), cache,
                         q_norm=None if not norm else norms[0].to(dev), k_norm=None if not norm else norms[1].to(dev), eps=1e-5,
                         out=None)
    assert got.dtype == torch.bfloat16 and got.shape == parts[0].shape
    want, slack = ref.turned(q, positions, freqs, inter, factor, norms[0], 1e-5)
    assert ref.bf16_close(got.cpu().view(T, Hq, D), want, slack).all()
    kw, ks = ref.turned(k, positions, freqs, inter, factor, norms[1], 1e-5)
    for held, x, s, scale in ((cache.k, kw, ks, cache.k_scale), (cache.v, v.double(), torch.zeros_like(ks), cache.v_scale)):
        held = held.cpu().float().transpose(1, 2).reshape(pages * page, Hkv, D)
        live = slots >= 0
        mine = held[slots[live].long()]
        if kind == "e4m3":
            f = scale.cpu().double()[:, None]
            assert ref.e4m3_close(mine, x[live] / f, s[live] / f + (x[live] / f).abs() * ref.EPS32).all()
        else:
            assert ref.bf16_close(mine, x[live], s[live]).all()
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[slots[live].long()] = False
        assert (held[rest] == 0).all()


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_types_layouts(dev, ty, kind, D, inter):
    check(dev, 37, 6, 2, D, D, ty, kind, inter=inter, norm=inter, seed=1)
    check(dev, 5, 3, 1, D, D // 2, ty, kind, inter=inter, norm=not inter, page=64, seed=2)


@pytest.mark.parametrize("R", [2, 4, 6, 32, 34, 66, 96, 126, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_part_of_the_head(dev, R, inter):
    check(dev, 9, 4, 2, 128, R, inter=inter, norm=True, seed=R)


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 32, 8), (2, 40, 8), (3, 7, 7), (64, 5, 1), (515, 14, 2), (1, 128, 16)])
def test_sizes(dev, T, Hq, Hkv):
    check(dev, T, Hq, Hkv, 128, 128, norm=True, seed=T, fused=False)
    check(dev, T, Hq, Hkv, 64, 64, torch.bfloat16, "e4m3", page=128, seed=T + 1)


@pytest.mark.parametrize("far", [1, 1 << 20, (1 << 31) - 1])
def test_far_positions(dev, far):
    check(dev, 40, 4, 2, 128, 128, far=far, factor=1.25, seed=3)


def test_negative_positions(dev):
    x = torch.randn(2, 1, 64)
    freqs = torch.rand(32)
    positions = torch.tensor([-7, -(1 << 31)], dtype=torch.int32)
    got = ql.rope_append(*(x.to(dev),) * 3, positions.to(dev), torch.tensor([-1, -1], dtype=torch.int32, device=dev),
                         ql.Rope(freqs.to(dev)), empty_cache(1, 1, 16, 64, "bf16", dev))
    want, slack = ref.turned(x, positions, freqs, False, 1.0, None, 0.0)
    assert ref.bf16_close(got.cpu(), want, slack).all()


def test_slots_outside_the_cache_and_pads(dev):
    """Only the slots that exist are written; q is turned for every row."""
    T, page, pages = 8, 16, 3
    cache = empty_cache(pages, 1, page, 64, "bf16", dev, fill=7.0)
    x = torch.randn(T, 1, 64)
    slots = torch.tensor([-1, pages * page, 2 ** 31 - 1, -(2 ** 31), 47, 0, pages * page + 5, 16], dtype=torch.int32)
    positions = torch.arange(T, dtype=torch.int32)
    freqs = torch.rand(32)
    got = ql.rope_append(*(x.to(dev),) * 3, positions.to(dev), slots.to(dev), ql.Rope(freqs.to(dev)), cache)
    want, slack = ref.turned(x, positions, freqs, False, 1.0, None, 0.0)
    assert ref.bf16_close(got.cpu(), want, slack).all()
    held = cache.v.cpu().view(pages * page, 64)
    for i, s in enumerate(slots.tolist()):
        if s in (47, 0, 16):
            assert torch.equal(held[s], x[i, 0].to(torch.bfloat16))
            held[s] = 7.0
    assert (held == 7.0).all()


def test_special_values(dev):
    """Infinities and NaN come through; e4m3 saturates and keeps NaN; a head of zeros stays zero under the norm."""
    nan, inf = float("nan"), float("inf")
    x = torch.zeros(4, 1, 64)
    x[0, 0, 40], x[1, 0, 3], x[2, 0, 50] = inf, nan, 1e30
    freqs = torch.zeros(32)  # cos 1, sin 0
    cache = empty_cache(1, 1, 16, 64, "e4m3", dev)
    pos = torch.zeros(4, dtype=torch.int32, device=dev)
    slots = torch.arange(4, dtype=torch.int32, device=dev)
    ql.rope_append(*(x.to(dev),) * 3, pos, slots, ql.Rope(freqs.to(dev)[:1]), cache)
    v = cache.v.cpu().float()[0, 0]
    assert v[0, 40] == 448 and torch.isnan(v[1, 3]) and v[2, 50] == 448 and (v[3] == 0).all()
    one = torch.ones(64, device=dev)
    q = ql.rope_append(*(x.to(dev),) * 3, pos, slots, ql.Rope(freqs.to(dev)), cache, q_norm=one, k_norm=one)
    assert (q[3] == 0).all() and torch.isnan(q[1]).all()


def test_into_given_memory_and_strides(dev):
    """Rows at any distance; nothing but out and the slots is written."""
    T, Hq, D = 6, 4, 128
    wide = torch.randn(2 * T, 3 * Hq * D + 64, device=dev)
    q, k, v = (wide[::2, i * Hq * D : (i + 1) * Hq * D] for i in range(3))
    freqs = torch.rand(D // 2, device=dev)
    pos = torch.arange(2 * T, dtype=torch.int32, device=dev)[3 : 3 + T]  # 4-byte aligned only
    slots = torch.arange(1, T + 1, dtype=torch.int32, device=dev)
    buf = torch.full((T * Hq * D + 128,), -3.0, dtype=torch.bfloat16, device=dev)
    out = buf[64:-64].view(T, Hq * D)
    c1, c2 = (empty_cache(1, Hq, 16, D, "bf16", dev) for _ in "ab")
    assert ql.rope_append(q, k, v, pos, slots, ql.Rope(freqs), c1, out=out) is out
    want = ql.rope_append(*(x.contiguous().view(T, Hq, D) for x in (q, k, v)), pos.clone(), slots, ql.Rope(freqs), c2)
    assert torch.equal(out, want.view(T, -1)) and torch.equal(c1.k, c2.k) and torch.equal(c1.v, c2.v)
    assert (buf[:64] == -3).all() and (buf[-64:] == -3).all()


def test_offsets_beyond_32_bits(dev):
    """A cache of more than 4 GiB: its last slots are written, its first are not."""
    pages, Hkv, page, D = 2100, 8, 1024, 128
    store = [torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device=dev) for _ in "kv"]
    cache = ql.KvCache(*store)
    assert 2 * pages * Hkv * page * D > 1 << 32
    x = torch.randn(2, Hkv, D, device=dev)
    slots = torch.tensor([pages * page - 1, pages * page - page - 2], dtype=torch.int32, device=dev)
    ql.rope_append(x, x, x, torch.zeros(2, dtype=torch.int32, device=dev), slots, ql.Rope(torch.ones(1, device=dev)), cache)
    want = x.to(torch.bfloat16)
    for t in (cache.k, cache.v):
        assert torch.equal(t[-1, :, -1], want[0]) and torch.equal(t[-2, :, -2], want[1])
        assert int((t != 0).sum()) == int((want != 0).sum())


def test_frequencies_by_parts(dev):
    f, factor = ql.rope_frequencies(128, 1e6, stretch=4.0, original=32768)
    check_f = ql.Rope(f.to(dev), factor=factor)
    x = torch.randn(3, 2, 128)
    pos = torch.tensor([0, 40000, 131071], dtype=torch.int32)
    got = ql.rope_append(*(x.to(dev),) * 3, pos.to(dev), torch.full((3,), -1, dtype=torch.int32, device=dev), check_f,
                         empty_cache(1, 2, 16, 128, "bf16", dev))
    want, slack = ref.turned(x, pos, f, False, factor, None, 0.0)
    assert ref.bf16_close(got.cpu(), want, slack).all()
    assert math.isclose(factor, 0.1 * math.log(4) + 1)
