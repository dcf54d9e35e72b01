"""Every compiled form of the experts' kernels, bit for bit.  Gates are at least 32, where silu(g) = g in fp32, and
sums are exact, so every hidden value gate * up is known: up to 24 bits, all of the three planes it is kept in."""
import pytest
import torch

import mx4_cases as cases
import mx4_plans as plans
from decode_gemv_thinkbit_amd import qlinear as ql

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ql.lib()
    return torch.device("cuda:0")


def route(T, k, E, g, dev, dropped=0.1):
    """k different experts of each token, some of them left out."""
    ids = torch.rand(T, E, generator=g, device=dev).argsort(1)[:, :k].int()
    return torch.where(torch.rand(T, k, generator=g, device=dev) < dropped, -1, ids)


def hidden(x, ids, gate, up):
    """gate * up in fp64 for every pair [T, k, I], 0 for pairs without an expert; checked to be exact in fp32."""
    T, k = ids.shape
    xs, h = x.double(), torch.zeros(T, k, gate.N, dtype=torch.float64, device=x.device)
    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        t, j = (ids == e).nonzero(as_tuple=True)
        one = [cases.values(ql.Mx4Tensor(w.codes[e].clone(), w.scales[e].clone())) for w in (gate, up)]
        a, b = (cases.exact_product(xs[t], w, 0.25) for w in one)
        assert float(a.min()) >= 32
        h[t, j] = a * b
    assert torch.equal(h, h.float().double())
    return h


def gate_up(E, H, I, T, g, dev):
    """Stacks and tokens: input 0 alone makes every gate large, the others are random of both signs, scaled so that
    the products fill 24 bits."""
    gate, up = (torch.randint(0, 16, (E, I, H), generator=g, device=dev, dtype=torch.uint8) for _ in range(2))
    x = torch.randint(-1, 2, (T, H), generator=g, device=dev)
    x = torch.where(torch.rand(T, H, generator=g, device=dev) < min(1.0, 128 / H), x, 0)
    most = next(m for m in (128, 64, 32, 16, 8, 4, 2, 1) if m * max(float(x.abs().sum(1).max()), 1.0) <= 128)
    x = (x * most).double()
    x[:, 0] = 256.0
    gate[..., 0], up[..., 0] = 7, 0
    scales = [torch.randint(125, 128, (E, I, 4 * ((H + 127) // 128)), generator=g, device=dev, dtype=torch.uint8)
              for _ in range(2)]
    scales[0][..., 0] = 127
    return x.bfloat16(), cases.mx4(gate, scales[0]), cases.mx4(up, scales[1])


@pytest.mark.parametrize("T,k,E,H,I", cases.MOE)
def test_hidden_values_one_by_one(dev, T, k, E, H, I):
    """Rows of the down projection with a single code: outputs are hidden values times powers of two."""
    g = torch.Generator(device=dev).manual_seed(T * 31 + k * 7 + E + H + I)
    x, gate, up = gate_up(E, H, I, T, g, dev)
    ids = route(T, k, E, g, dev)
    h = hidden(x, ids, gate, up)
    lowest = torch.where(h != 0, h.abs().log2().floor() - 7, 0.0)  # of the eight bits that one plane holds
    assert T * I < 500 or (torch.remainder(h, torch.exp2(lowest)) != 0).float().mean() > 0.3
    assert T * I < 5000 or (torch.remainder(h, torch.exp2(lowest - 9)) != 0).any()  # past two planes
    rows = torch.arange(H, device=dev)
    for shift in range(0, min(I, 3 * H), H):
        column = (rows + shift) % I
        code = torch.randint(0, 4, (E, H), generator=g, device=dev)
        codes = torch.zeros(E, H, I, dtype=torch.uint8, device=dev)
        codes[:, rows, column] = torch.tensor([1, 2, 4, 6], dtype=torch.uint8, device=dev)[code]  # 0.5, 1, 2, 4
        codes[:, rows, column] |= (torch.randint(0, 2, (E, H), generator=g, device=dev) * 8).to(torch.uint8)
        scales = torch.randint(100, 140, (E, H, 4 * ((I + 127) // 128)), generator=g, device=dev, dtype=torch.uint8)
        down = cases.mx4(codes, scales)
        factor = torch.exp2(code.double() - 1 + scales[:, rows, column // 32].double() - 127)
        factor = torch.where(codes[:, rows, column] >= 8, -factor, factor)
        for slot in range(k):  # the others carry no weight
            weights = torch.zeros(T, k, device=dev)
            weights[:, slot] = 1.0
            y = ql.mx4_moe(x, ids, weights, gate, up, down)
            e = ids[:, slot].long().clamp(min=0)
            want = h[:, slot][:, column] * factor[e] * (ids[:, slot] >= 0).double()[:, None]
            assert torch.equal(y.double(), want), (shift, slot, int((y.double() != want).sum()), y.numel())


@pytest.mark.parametrize("T,k,E,H,I", cases.MOE)
def test_whole_rows(dev, T, k, E, H, I):
    """Full rows of the down projection and small hidden values: sums are exact, a block left out or taken twice
    shows."""
    check_whole_rows(T, k, E, H, I, None, dev)


def check_whole_rows(T, k, E, H, I, ids, dev):
    g = torch.Generator(device=dev).manual_seed(T * 13 + k * 5 + E + H + I)
    few = lambda *s: torch.rand(*s, generator=g, device=dev) < 6 / H
    gate, up = (torch.where(few(E, I, H), torch.randint(0, 16, (E, I, H), generator=g, device=dev) & 10, 0).to(torch.uint8)
                for _ in range(2))  # 0, 1 and their negatives
    gate[..., 0], up[..., 0] = 7, 0
    x = torch.randint(-1, 2, (T, H), generator=g, device=dev).double()
    x[:, 0] = 8.0
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device=dev)
    stride = lambda n: 4 * ((n + 127) // 128)
    gate, up = (cases.mx4(c, one(E, I, stride(H))) for c in (gate, up))
    down = cases.mx4((torch.randint(0, 3, (E, H, I), generator=g, device=dev)
                      + 8 * torch.randint(0, 2, (E, H, I), generator=g, device=dev)).to(torch.uint8), one(E, H, stride(I)))
    if ids is None:
        ids = route(T, k, E, g, dev)
    weights = torch.tensor([1.0, -1.0, 0.5, 2.0], device=dev)[torch.randint(0, 4, (T, k), generator=g, device=dev)]
    h = hidden(x, ids, gate, up)
    want, size = (torch.zeros(T, H, dtype=torch.float64, device=dev) for _ in range(2))
    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        t, j = (ids == e).nonzero(as_tuple=True)
        d = cases.values(ql.Mx4Tensor(down.codes[e].clone(), down.scales[e].clone()))
        want.index_add_(0, t, cases.exact_product(h[t, j], d, 0.5) * weights[t, j].double()[:, None])
        size.index_add_(0, t, (h[t, j].abs() @ d.abs().t().contiguous()) * weights[t, j].abs().double()[:, None])
    assert float(size.max()) < 2 ** 24 * 0.25
    y = ql.mx4_moe(x.bfloat16(), ids, weights, gate, up, down)
    assert torch.equal(y.double(), want), (int((y.double() != want).sum()), y.numel())


def test_shared_tasks_in_a_second_round(dev):
    """The kernel that shares a task among four waves, with more tasks than workgroups run at a time: for it, groups
    of two pairs (three pairs an expert make two groups), and of four."""
    ids = torch.tensor([e for e in range(10) for _ in range(3)] + [-1, 15], dtype=torch.int32, device=dev).view(2, 16)
    (xp, waves, join, small, tail), _ = plans.moe(2, 16, 16, 256, 1024)
    assert join and xp == 1 and (2 * 10 + 1) * 1024 // 16 > 4 * 256
    check_whole_rows(2, 16, 16, 256, 1024, ids, dev)
    ids = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7], [8, 9]], dtype=torch.int32, device=dev)
    (xp, waves, join, small, tail), _ = plans.moe(5, 2, 10, 256, 1600)
    assert join and xp == 2 and 10 * 1600 // 16 > 3 * 256
    check_whole_rows(5, 2, 10, 256, 1600, ids, dev)
