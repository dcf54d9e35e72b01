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
