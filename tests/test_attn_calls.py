"""What the binding of the rotary and attention operators passes on, and what it keeps alive (CPU only; the launches
are stubs)."""
import weakref

import pytest
import torch

from decode_gemv_thinkbit_amd import qlinear as ql


def zeros(*s, t=torch.bfloat16):
    return torch.zeros(*s, dtype=t)


def ints(*s):
    return torch.zeros(*s, dtype=torch.int32)


@pytest.fixture
def launches(monkeypatch):
    """The launches' arguments, host tensors let through."""
    ran = []
    monkeypatch.setattr(ql, "_launch", lambda what, fn, device, *args: ran.append((what, args)))
    check = ql._cache

    class Gpu:  # what the check of the device looks at
        type = "cuda"

        def __init__(self, device):
            self.device = device

        def __eq__(self, other):
            return self.device == other

        __hash__ = None

    monkeypatch.setattr(ql, "_cache", lambda cache, device: check(cache, Gpu(device)))
    monkeypatch.setattr(ql, "_workspace_bytes", lambda *sizes: 64)
    return ran


def cache(pages=3):
    return ql.KvCache(zeros(pages, 2, 16, 64), zeros(pages, 2, 16, 64))


@pytest.mark.parametrize("call", [lambda c: ql.attn_decode(zeros(1, 4, 64), c, ints(1, 3), ints(1)),
                                  lambda c: ql.attn_prompt(zeros(1, 4, 64), ints(2), c, ints(1, 3), ints(1))])
def test_a_workspace_lives_until_the_launch(launches, monkeypatch, call):
    """Given back before it, another thread could get it and come between the two kernels, or have it unmapped."""
    made, alive = [], []

    def scratch(workspace, need, device):
        t = torch.empty(need, dtype=torch.uint8)
        made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(ql, "_scratch", scratch)
    monkeypatch.setattr(ql, "_launch", lambda what, fn, device, *args: alive.append(made[-1]() is not None))
    call(cache())
    assert alive == [True]


def rope_call(c, rope):
    ql.rope_append(zeros(1, 4, 64), zeros(1, 2, 64), zeros(1, 2, 64), ints(1), ints(1), rope, c)


CALLS = [lambda c: rope_call(c, ql.Rope(torch.ones(32))), lambda c: ql.attn_decode(zeros(1, 4, 64), c, ints(1, 3), ints(1)),
         lambda c: ql.attn_prompt(zeros(1, 4, 64), ints(2), c, ints(1, 3), ints(1))]


def passed(args, of):
    """The struct `of` among a launch's arguments, which are packed descriptors, numbers and addresses."""
    import ctypes

    return next(of.from_buffer_copy(a) for a in args if isinstance(a, bytes) and len(a) == ctypes.sizeof(of))


def grown(t):
    t.untyped_storage().resize_(8 * t.untyped_storage().nbytes())


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("move", [lambda t: t.set_(torch.ones_like(t)), lambda t: setattr(t, "data", torch.ones_like(t)), grown])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_cache_is_where_its_tensors_are_now(launches, call, move, kind):
    """Tensors that were given other memory are used there: what they had may belong to another."""
    scales = [torch.ones(2) for _ in "kv"] if kind != torch.bfloat16 else []
    c = ql.KvCache(*(torch.zeros(3, 2, 16, 64).to(kind) for _ in "kv"), *scales)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        if t is None:
            continue
        held = t.data_ptr()
        keep = t.untyped_storage() if move is not grown else None
        move(t)
        assert move is grown or t.data_ptr() != held
        call(c)
        d = passed(launches[-1][1], ql.ql_kv_cache)
        want = [x if x is None else x.data_ptr() for x in (c.k, c.v, c.k_scale, c.v_scale)]
        assert [d.k, d.v, d.k_scale, d.v_scale] == want
        del keep


def test_a_rope_is_where_its_frequencies_are_now(launches):
    rope, c = ql.Rope(torch.ones(32)), cache()
    first = rope.freqs.untyped_storage()
    rope.freqs.data = torch.rand(16)
    rope_call(c, rope)
    d = passed(launches[-1][1], ql.ql_rope)
    assert (d.freqs, d.dims) == (rope.freqs.data_ptr(), 32)
    del first


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("other", [zeros(3, 2, 16, 128), zeros(3, 2, 16, 64, t=torch.float32), zeros(3, 16, 2, 64).transpose(1, 2),
                                   zeros(0)])
def test_a_cache_that_no_longer_fits_is_refused(launches, call, other):
    c = cache()
    c.k.data = other
    with pytest.raises(ValueError):
        call(c)
    with pytest.raises(ValueError):  # and the next time
        call(c)
    assert not launches


def test_a_cache_follows_its_tensors_shape(launches):
    c = cache()
    for t in (c.k, c.v):
        t.data = zeros(5, 1, 32, 128)
    ql.attn_decode(zeros(1, 4, 128), c, ints(1, 3), ints(1))
    d = passed(launches[-1][1], ql.ql_kv_cache)
    assert (d.pages, d.heads, d.page, d.dim) == (5, 1, 32, 128)


@pytest.mark.parametrize("T,B,Hq,Hkv,D,keys", [(64, 64, 32, 8, 128, 8192), (256, 64, 32, 8, 128, 8192), (256, 256, 32, 8, 128, 8192),
                                               (70, 70, 32, 8, 128, 131072), (2048, 2048, 8, 8, 128, 8192), (16384, 16384, 1, 1, 128, 8192),
                                               (1, 1, 32, 8, 128, 131072), (9, 1, 128, 1, 64, 1 << 20), (300, 7, 40, 8, 128, 32768),
                                               (5, 3000, 32, 8, 128, 4096), (1025, 1025, 14, 2, 64, 65536)])
def test_a_prompts_workspace_is_for_its_rows(T, B, Hq, Hkv, D, keys):
    """Parts hold the rows that there are, not a tile of 128 for each sequence (1072 MiB for 64 sequences of one): the rows
    that are split fill at most 512 tiles of 128, each of D sums and two numbers."""
    need = ql.lib().qlinear_attn_prompt_workspace_bytes(T, B, Hq, Hkv, D, keys)
    assert 0 < need <= 512 * 128 * (D + 2) * 4 and need % (T * Hq * (D + 2) * 4) == 0


@pytest.mark.parametrize("strides", [dict(qs=1), dict(ks=1, vs=3), dict(qs=0, ks=0, vs=0), dict(dtype=1, qs=1 << 40)])
def test_a_single_row_has_no_stride(strides):
    """No distance is taken from it: a tensor of one row may have any (torch.empty(N, 1).t() is contiguous)."""
    import test_attn as calls

    assert calls.rope_call(T=1, out=calls.ODD, **strides) == 1 and "aligned" in calls.message(), calls.message()
