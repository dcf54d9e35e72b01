"""Attention over caches so long that they are cut into many parts: every part of them counts once (GPU)."""
import pytest
import torch

import attn_marks as marks
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


def on(dev, vs, page, kind, seed=0):
    (k, v), table = marks.cache_of(vs, page, kind, seed=seed)
    scales = [torch.full((k.shape[1],), 0.5, device=dev) for _ in "kv"] if kind == "e4m3" else []
    return ql.KvCache(k.to(dev), v.to(dev), *scales), table.to(dev)


# Lengths, kv heads, heads.  Rows of one slice and of four (tables of more than 16384 tokens and fewer than 256 rows), of more
# parts and of fewer than their joining reads ahead, parts of 128 keys and of several times that.
LONG = [([65536], 1, 2), ([65536], 8, 32), ([20011, 3, 0, 513], 1, 4), ([16300], 1, 1), ([16000, 9000], 2, 4), ([40000, 300] * 4, 2, 64),
        ([131072], 4, 4)]


@pytest.mark.parametrize("lens,Hkv,Hq", LONG)
@pytest.mark.parametrize("D,kind", [(64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "e4m3")])
def test_decode_counts_every_part_once(dev, lens, Hkv, Hq, D, kind):
    """Equal scores: each dim of the output is a count of tokens."""
    q = torch.zeros(len(lens), Hq, D, dtype=torch.bfloat16, device=dev)
    for at in (None, 0, 31, 32, 127):
        vs = [marks.blocks(n, 128, D, at).unsqueeze(1).repeat(1, Hkv, 1) for n in lens]
        cache, table = on(dev, vs, 64, kind)
        got = ql.attn_decode(q, cache, table, ints(lens, dev)).cpu()
        for b, v in enumerate(vs):
            want = marks.equal_weights(v[:, 0]) if lens[b] else torch.zeros(D, dtype=torch.float64)
            assert marks.close(got[b], want).all(), (at, b)


@pytest.mark.parametrize("new,before,Hkv,Hq", [([16], [65536 - 16], 1, 4), ([1], [40000], 8, 32), ([3, 0, 40], [20000, 5, 700], 2, 8),
                                               ([300], [9000], 8, 8), ([200], [16384], 2, 8)])
@pytest.mark.parametrize("D,kind", [(64, "bf16"), (128, "bf16"), (128, "e4m3")])
def test_prompts_count_every_part_once(dev, new, before, Hkv, Hq, D, kind):
    lens = [n + p for n, p in zip(new, before)]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    q = torch.zeros(starts[-1], Hq, D, dtype=torch.bfloat16, device=dev)
    for at in (None, 0, 31, 63):
        vs = [marks.blocks(n, 64, D, at).unsqueeze(1).repeat(1, Hkv, 1) for n in lens]
        cache, table = on(dev, vs, 64, kind)
        got = ql.attn_prompt(q, ints(starts, dev), cache, table, ints(lens, dev)).cpu()
        for b, v in enumerate(vs):
            sums = v[:, 0].double().cumsum(0)
            for i in range(0, new[b], 1 + new[b] // 9):
                sees = before[b] + i + 1
                assert marks.close(got[starts[b] + i], sums[sees - 1] / sees).all(), (at, b, i)


@pytest.mark.parametrize("lens,Hkv,Hq", [([65536], 1, 2), ([20011, 3, 0, 513], 1, 4), ([16300], 2, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_weighs_every_part(dev, lens, Hkv, Hq, D):
    """Scores of their own for each token: a dim is the weight of its blocks' tokens."""
    vs = [marks.blocks(n, 128, D).unsqueeze(1).repeat(1, Hkv, 1) for n in lens]
    cache, table = on(dev, vs, 64, "bf16", seed=3)
    q = ref.queries(len(lens), Hq, D, 4)
    got = ql.attn_decode(q.to(dev), cache, table, ints(lens, dev)).cpu()
    k_host = cache.k.cpu()
    for b, v in enumerate(vs):
        n = lens[b]
        if not n:
            continue
        k = k_host[table[b, : -(-n // 64)].cpu().long()].transpose(1, 2).reshape(-1, Hkv, D)[:n].double()
        want, slack = ref.attention(q[b : b + 1], k, v.double(), torch.ones(1, n, dtype=torch.bool), D ** -0.5)
        assert (slack <= 0.03 * want).all()  # where a block of 128 tokens is an eighth or more of a dim
        assert ref.bf16_close(got[b : b + 1], want, slack).all(), b
