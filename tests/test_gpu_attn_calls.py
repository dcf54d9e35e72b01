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
