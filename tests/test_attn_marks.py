"""The marked values of the long-cache tests show what they are meant to show (CPU only)."""
import pytest
import torch

import attn_marks as marks


@pytest.mark.parametrize("n,D", [(65536, 64), (65536, 128), (20011, 64), (9000, 128)])
@pytest.mark.parametrize("step,at", [(128, None), (128, 0), (128, 127), (64, 31)])
def test_a_part_left_out_or_taken_twice_is_seen(n, D, step, at):
    v = marks.blocks(n, step, D, at)
    want = marks.equal_weights(v)
    assert marks.close(want.to(torch.bfloat16), want).all()
    for first in range(0, n - step, 997 * step // 16):
        first = first // step * step
        part = v[first : first + step].double().sum(0)
        for sign in (-1, 1):  # of all sums, the divisor among them, and of the values alone
            assert not marks.close(((v.double().sum(0) + sign * part) / (n + sign * step)).to(torch.bfloat16), want).all()
            assert not marks.close(((v.double().sum(0) + sign * part) / n).to(torch.bfloat16), want).all()


def test_a_token_at_a_blocks_end_is_seen():
    n, D = 65536, 64
    for at in (0, 127):
        v = marks.blocks(n, 128, D, at)
        want = marks.equal_weights(v)
        for block in range(0, n // 128, 37):
            lost = v.double().sum(0)
            lost[block % D] -= 1
            assert not marks.close((lost / (n - 1)).to(torch.bfloat16), want).all()


def test_pages_hold_the_marks():
    vs = [marks.blocks(n, 128, 64).unsqueeze(1).repeat(1, 2, 1) for n in (300, 0, 17)]
    (k, v), table = marks.cache_of(vs, 16, "bf16")
    for b, x in enumerate(vs):
        n = x.shape[0]
        rows = table[b, : -(-n // 16)].long()
        assert torch.equal(v[rows].transpose(1, 2).reshape(-1, 2, 64)[:n].float(), x)
