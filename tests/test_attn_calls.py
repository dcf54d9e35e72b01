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
