"""The rotary and attention entry points refuse what they cannot do before anything reaches the GPU, their
sizes, and the frequencies of long contexts (CPU only)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attn_reference as ref
from decode_gemv_thinkbit_amd import qlinear as ql

FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation first
ODD = 0x10008
BAD = 0x10002


def message():
    return ql.lib().qlinear_last_error().decode()


def cache(**change):
    c = dict(pages=8, heads=2, page=16, dim=128, type=1, k=FAKE, v=FAKE, k_scale=None, v_scale=None)
    c.update(change)
    return ql.ql_kv_cache(c["pages"], c["heads"], c["page"], c["dim"], c["type"], 0, c["k"], c["v"], c["k_scale"], c["v_scale"])


CACHES = [(dict(pages=0), "pages"), (dict(pages=1 << 27), "pages"), (dict(heads=0), "heads"), (dict(heads=3), "heads"),
          (dict(heads=5000), "heads"), (dict(page=8), "page"), (dict(page=48), "page"), (dict(page=8192), "page"),
          (dict(page=-16), "page"), (dict(dim=96), "dim"), (dict(dim=256), "dim"), (dict(type=0), "type"), (dict(type=2), "type"),
          (dict(k=None), "null"), (dict(v=ODD), "aligned"), (dict(k_scale=FAKE), "no scales"), (dict(type=3), "null"),
          (dict(type=3, k_scale=FAKE, v_scale=BAD), "aligned")]


def rope_call(c=None, rope=None, **change):
    a = dict(T=4, Hq=8, dtype=0, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, pos=FAKE, slots=FAKE, qn=None, kn=None, eps=1e-6,
             out=FAKE)
    a.update(change)
    c = cache() if c is None else c
    rope = ql.ql_rope(FAKE, 128, 0, 1.0, 0) if rope is None else rope
    return ql.lib().qlinear_rope_append(a["T"], a["Hq"], a["dtype"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"],
                                        a["slots"], ctypes.byref(rope), a["qn"], a["kn"], a["eps"], ctypes.byref(c), a["out"], None)


def decode_call(c=None, **change):
    a = dict(B=4, Hq=8, q=FAKE, table=FAKE, stride=9, most=9, lens=FAKE, scale=0.1, out=FAKE, ws=FAKE, bytes=0)
    a.update(change)
    c = cache() if c is None else c
    return ql.lib().qlinear_attn_decode(ctypes.byref(c), a["B"], a["Hq"], a["q"], a["table"], a["stride"], a["most"], a["lens"],
                                        a["scale"], a["out"], a["ws"], a["bytes"], None)


def prompt_call(c=None, **change):
    a = dict(T=16, B=4, Hq=8, q=FAKE, starts=FAKE, table=FAKE, stride=900, most=900, lens=FAKE, scale=0.1, out=FAKE, ws=FAKE, bytes=0)
    a.update(change)
    c = cache() if c is None else c
    return ql.lib().qlinear_attn_prompt(ctypes.byref(c), a["T"], a["B"], a["Hq"], a["q"], a["starts"], a["table"], a["stride"],
                                        a["most"], a["lens"], a["scale"], a["out"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("change,word", CACHES)
def test_cache_refusals(change, word):
    for call in (rope_call, decode_call, prompt_call):
        assert call(cache(**change)) == 1 and word in message(), message()


@pytest.mark.parametrize("change,word", [
    (dict(T=0), "T"), (dict(T=1 << 24), "T"), (dict(Hq=0), "heads"), (dict(Hq=7), "heads"), (dict(dtype=3), "type"),
    (dict(dtype=-1), "type"), (dict(q=None), "null"), (dict(k=ODD), "aligned"), (dict(qs=1023), "stride"), (dict(qs=1026), "stride"),
    (dict(ks=252), "stride"), (dict(dtype=1, vs=260), "stride"), (dict(qs=-1024), "stride"), (dict(pos=None), "null"), (dict(slots=BAD), "4-byte"),
    (dict(qn=BAD), "4-byte"), (dict(eps=-1.0), "eps"), (dict(eps=math.nan), "eps"), (dict(eps=math.inf), "eps"), (dict(out=ODD), "aligned"),
    (dict(rope=ql.ql_rope(FAKE, 0, 0, 1.0, 0)), "dims"), (dict(rope=ql.ql_rope(FAKE, 130, 0, 1.0, 0)), "dims"),
    (dict(rope=ql.ql_rope(FAKE, 63, 0, 1.0, 0)), "dims"), (dict(rope=ql.ql_rope(None, 64, 0, 1.0, 0)), "null"),
    (dict(rope=ql.ql_rope(FAKE, 64, 0, math.nan, 0)), "factor")])
def test_rope_refusals(change, word):
    assert rope_call(**change) == 1 and word in message(), message()


COMMON = [(dict(B=0), "B"), (dict(B=1 << 24), "B"), (dict(Hq=9), "heads"), (dict(q=None), "null"), (dict(q=ODD), "aligned"),
          (dict(out=ODD), "aligned"), (dict(table=None), "null"), (dict(lens=BAD), "4-byte"), (dict(scale=0.0), "scale"),
          (dict(scale=-1.0), "scale"), (dict(scale=math.nan), "scale"), (dict(scale=math.inf), "scale"), (dict(most=0), "table"),
          (dict(stride=8), "table"), (dict(most=1 << 27, stride=1 << 27), "tokens"),
          (dict(most=(1 << 26) + 1, stride=(1 << 26) + 1), "tokens")]


@pytest.mark.parametrize("change,word", COMMON + [(dict(B=1 << 21, stride=9), "too many"), (dict(most=900, stride=900), "workspace"),
                                                  (dict(most=900, stride=900, bytes=1 << 40, ws=None), "null"),
                                                  (dict(most=900, stride=900, bytes=1 << 40, ws=ODD), "aligned")])
def test_decode_refusals(change, word):
    assert decode_call(**change) == 1 and word in message(), message()


@pytest.mark.parametrize("change,word", COMMON + [(dict(T=0), "T"), (dict(T=1 << 24), "T"), (dict(starts=None), "null"), (dict(starts=BAD), "4-byte"),
                                                  (dict(T=1 << 23, Hq=256), "T \\* Hq"), (dict(B=1 << 23), "too many"),
                                                  (dict(), "workspace"), (dict(bytes=1 << 40, ws=None), "null"),
                                                  (dict(bytes=1 << 40, ws=ODD), "aligned")])
def test_prompt_refusals(change, word):
    assert prompt_call(**change) == 1 and word.replace("\\", "") in message(), message()


def test_null_structs():
    L = ql.lib()
    assert L.qlinear_attn_decode(None, 1, 1, FAKE, FAKE, 1, 1, FAKE, 1.0, FAKE, None, 0, None) == 1 and "cache" in message()
    c = cache()
    assert L.qlinear_rope_append(4, 8, 0, FAKE, 1024, FAKE, 256, FAKE, 256, FAKE, FAKE, None, None, None, 1e-6, ctypes.byref(c),
                                 FAKE, None) == 1 and "rope" in message()


def test_packed_descriptors_are_the_structs():
    """The binding packs what the header declares."""
    for pack, of, values in ((ql._pack_cache, ql.ql_kv_cache, (8, 2, 16, 128, 3, 0, FAKE, ODD, BAD, FAKE)),
                             (ql._pack_rope, ql.ql_rope, (FAKE, 64, 1, 1.25, 0))):
        raw = pack(*values)
        assert len(raw) == ctypes.sizeof(of)
        held = of.from_buffer_copy(raw)
        assert tuple(getattr(held, f) for f, _ in of._fields_) == values


def test_workspace_sizes():
    L = ql.lib()
    assert L.qlinear_attn_decode_workspace_bytes(4, 8, 2, 128, 16) == 0  # one part
    assert L.qlinear_attn_decode_workspace_bytes(4, 8, 2, 96, 4096) == 0  # refused
    one, two = (L.qlinear_attn_decode_workspace_bytes(b, 32, 8, 128, 1 << 17) for b in (1, 64))
    assert 0 < one <= two < 1 << 28
    assert L.qlinear_attn_prompt_workspace_bytes(8192, 1, 32, 8, 128, 8192) == 0  # rows enough
    assert 0 < L.qlinear_attn_prompt_workspace_bytes(16, 1, 32, 8, 128, 1 << 17) < 1 << 30
    assert L.qlinear_attn_prompt_workspace_bytes(16, 1, 32, 7, 128, 1 << 17) == 0


def test_cache_checks():
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s).to(t)
    c = ql.KvCache(z(3, 2, 16, 64), z(3, 2, 16, 64))
    assert c.shape == (3, 2, 16, 64) and c.nbytes == 2 * 3 * 2 * 16 * 64 * 2
    with pytest.raises(AttributeError):  # its shape was checked
        c.k = z(1, 2, 16, 64)
    s = torch.ones(2)
    e = ql.KvCache(z(3, 2, 16, 64, t=ref.F8), z(3, 2, 16, 64, t=ref.F8), s, s)
    assert e.nbytes == c.nbytes // 2
    good = z(3, 2, 16, 64)
    for args in ((good, z(3, 2, 16, 128)), (good.float(), good.float()), (good, z(3, 2, 16, 64, t=ref.F8)), (z(3, 2, 16, 96),) * 2,
                 (z(3, 2, 8, 64),) * 2, (z(3, 2, 24, 64),) * 2, (z(0, 2, 16, 64),) * 2, (z(2, 16, 64),) * 2,
                 (z(3, 16, 2, 64).transpose(1, 2),) * 2, (good, good, s, s), (e.k, e.v), (e.k, e.v, s, None),
                 (e.k, e.v, s, torch.ones(3)), (e.k, e.v, s.double(), s.double())):
        with pytest.raises(ValueError):
            ql.KvCache(*args)
    for f in (torch.ones(4, dtype=torch.float64), torch.ones(2, 2), torch.ones(0), torch.ones(8)[::2]):
        with pytest.raises(ValueError):
            ql.Rope(f)


def test_binding_refuses_host_tensors_and_shapes():
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)
    c = ql.KvCache(z(3, 2, 16, 64), z(3, 2, 16, 64))
    i = lambda *s: z(*s, t=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ql.rope_append(z(1, 4, 64), z(1, 2, 64), z(1, 2, 64), i(1), i(1), ql.Rope(torch.ones(32)), c)
    with pytest.raises(ValueError, match="CUDA"):
        ql.attn_decode(z(1, 4, 64), c, i(1, 3), i(1))
    with pytest.raises(ValueError, match="CUDA"):
        ql.attn_prompt(z(1, 4, 64), i(2), c, i(1, 3), i(1))


# ---------------------------------------------------------------- frequencies
def test_frequencies():
    f, factor = ql.rope_frequencies(8, 10000.0)
    assert f.dtype == torch.float32 and factor == 1.0 and np.allclose(f.numpy(), [1, 0.1, 0.01, 0.001], rtol=2.0 ** -24)
    g, factor = ql.rope_frequencies(8, 10000.0, stretch=4.0)
    assert factor == 1.0 and torch.equal(g, f / 4)
    assert torch.equal(ql.rope_frequencies(8, 10000.0, stretch=1.0, original=100)[0], f)


def test_frequencies_by_parts():
    """Pairs that turn often within the original context are kept, slow ones stretched, between them a ramp."""
    dims, base, stretch, original = 128, 1e6, 4.0, 32768
    f, factor = ql.rope_frequencies(dims, base, stretch, original)
    plain = base ** (-2 * np.arange(dims // 2) / dims)
    turns = original * plain / (2 * np.pi)
    ratio = f.double().numpy() / plain
    assert np.allclose(ratio[turns > 33 * 1.3], 1, rtol=1e-6) and np.allclose(ratio[turns < 0.75], 0.25, rtol=1e-6)
    assert (np.diff(ratio) <= 1e-6).all() and ((ratio > 0.26) & (ratio < 0.99)).sum() > 3
    assert math.isclose(factor, 0.1 * math.log(4.0) + 1)


@pytest.mark.parametrize("args", [(7,), (0,), (8, 1.0), (8, 10.0, 0.5), (8, 10.0, 2.0, 0), (8, 10.0, 2.0, 100, 1.0, 1.0),
                                  (8, math.nan), (8, 10.0, math.nan)])
def test_frequency_refusals(args):
    with pytest.raises(ValueError):
        ql.rope_frequencies(*args)


# ---------------------------------------------------------------- the reference itself
def test_reference_pins():
    """One key: its value; equal scores: the mean; a rotation by a quarter turn."""
    k = torch.ones(2, 1, 64, dtype=torch.float64)
    v = torch.stack([torch.full((1, 64), 1.0), torch.full((1, 64), 3.0)]).double()
    q = torch.ones(1, 1, 64, dtype=torch.bfloat16)
    for sees, want in (([True, False], 1.0), ([True, True], 2.0), ([False, False], 0.0)):
        out, _ = ref.attention(q, k, v, torch.tensor([sees]), 0.125)
        assert torch.allclose(out, torch.full_like(out, want))
    x = torch.zeros(1, 1, 64)
    x[0, 0, 1], x[0, 0, 40] = 2.0, 5.0
    quarter = torch.full((32,), math.pi / 2)
    y, _ = ref.turned(x, torch.tensor([1]), quarter, False, 1.0, None, 0.0)
    assert abs(y[0, 0, 33] - 2) < 1e-6 and abs(y[0, 0, 8] + 5) < 1e-6 and abs(y[0, 0, 1]) < 1e-6
    y, _ = ref.turned(x, torch.tensor([1]), quarter, True, 1.0, None, 0.0)
    assert abs(y[0, 0, 0] + 2) < 1e-6 and abs(y[0, 0, 41] - 5) < 1e-6
