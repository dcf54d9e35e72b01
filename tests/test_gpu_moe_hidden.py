"""The hidden values silu(gate) * up of the experts' products, pinned one by one: inputs whose sums are exact give
known hidden values, and rows of the down projection with a single code give each of them back, bit for bit."""
import numpy as np
import pytest
import torch

from decode_gemv_thinkbit_amd import qlinear as ql

pytestmark = pytest.mark.gpu

CODE = {0.0: 0, 0.5: 1, 1.0: 2, 1.5: 3, 2.0: 4, 3.0: 5, 4.0: 6, 6.0: 7}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ql.lib()
    return torch.device("cuda:0")


def matrix(rows, K, entries, exponents, dev):
    """A stack of one [rows, K] matrix: entries {(row, input): value}, every scale of a row 2^exponents[row]."""
    c = np.zeros((rows, K), np.uint8)
    for (n, k), v in entries.items():
        c[n, k] = CODE[abs(v)] | (8 if v < 0 else 0)
    s = np.repeat(np.asarray(exponents, np.int64)[:, None] + 127, 4 * ((K + 127) // 128), 1)
    assert s.min() >= 0 and s.max() < 255
    return ql.Mx4Tensor(torch.from_numpy(c[:, 0::2] | c[:, 1::2] << 4)[None].contiguous().to(dev),
                        torch.from_numpy(s.astype(np.uint8))[None].contiguous().to(dev))


def hidden_through(x, gate, up, back, T, dev):
    """y [32] of T equal tokens through one expert whose down projection gives hidden value n times 2^back in row n."""
    down = matrix(32, 32, {(n, n): 1.0 for n in range(32)}, [back] * 32, dev)
    xs = torch.tensor(x, dtype=torch.float64).to(torch.bfloat16)
    assert torch.equal(xs.double(), torch.tensor(x, dtype=torch.float64))
    y = ql.mx4_moe(xs.repeat(T, 1).to(dev), torch.zeros(T, 1, dtype=torch.int32, device=dev),
                   torch.ones(T, 1, device=dev), gate, up, down)
    assert (y == y[0]).all()
    return y[0].cpu().double().numpy()


@pytest.mark.parametrize("T", [1, 2, 5, 64])
def test_values_that_round_past_the_largest_bf16(dev, T):
    """Finite hidden values between 2^128 (1 - 2^-9) and the largest fp32 stay finite."""
    x = [0.0] * 32
    x[:5] = [1.9921875, 1.0, 2.0 ** -9, 2.0 ** -10, 2.0 ** -8]
    ups = [{1: 1.0, 2: 1.0, 3: 1.0}, {1: 1.0, 4: 1.0}, {1: -1.0, 2: -1.0, 3: -1.0}, {1: -1.0, 4: -1.0}, {1: 1.0}]
    gate = matrix(32, 32, {(n, 0): 1.0 for n in range(32)}, [60] * 32, dev)
    up = matrix(32, 32, {(n, k): v for n in range(32) for k, v in ups[n % 5].items()}, [67] * 32, dev)
    h = np.array([x[0] * sum(v * x[k] for k, v in ups[n % 5].items()) for n in range(32)]) * 2.0 ** 127
    assert np.array_equal(h, h.astype(np.float32).astype(np.float64))  # exact in fp32
    assert (np.abs(h) > 2.0 ** 128 * (1 - 2.0 ** -9)).sum() > 20 and np.isfinite(h.astype(np.float32)).all()
    assert np.array_equal(hidden_through(x, gate, up, -20, T, dev), h * 2.0 ** -20)


@pytest.mark.parametrize("T", [1, 2, 5, 64])
def test_small_values_keep_their_bits_down_to_the_least_bf16(dev, T):
    """Hidden values below 2^-110 are kept to half of 2^-133."""
    x = [0.0] * 32
    x[:3] = [1.0, 2.0 ** -8, 2.0 ** -13]
    exponents = [-100 - n for n in range(28)] + [-100] * 4
    gate = matrix(32, 32, {(n, 0): 1.0 for n in range(32)}, [5] * 32, dev)
    up = matrix(32, 32, {(n, k): 1.0 if k < 2 else 1.5 for n in range(32) for k in range(3)}, exponents, dev)
    h = np.array([2.0 ** (5 + e) * (1 + 2.0 ** -8 + 1.5 * 2.0 ** -13) for e in exponents])
    assert (h < 2.0 ** -110).any() and (h % 2.0 ** -133 != 0).any()
    got = hidden_through(x, gate, up, 40, T, dev) * 2.0 ** -40
    assert (np.abs(got - h) <= 2.0 ** -134).all() and np.array_equal(got[h >= 2.0 ** -110], h[h >= 2.0 ** -110])


@pytest.mark.parametrize("T", [1, 2, 5, 64])
def test_silu_where_its_exponential_overflows(dev, T):
    """Gates below -88 with large up projections: exp(-g) is beyond fp32, silu(g) * u is not."""
    x = [0.0] * 32
    x[:4] = [80.0, 1.0, 8.0, 1.0]
    more = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    gate = matrix(32, 32, {(n, k): v for n in range(32) for k, v in ((0, -1.0), (1, -more[n % 8]), (2, -more[n // 4]))},
                  [0] * 32, dev)
    up = matrix(32, 32, {(n, 3): 1.0 if n % 3 else -1.0 for n in range(32)}, [100] * 32, dev)
    g = np.array([-80.0 - more[n % 8] - 8 * more[n // 4] for n in range(32)])
    h = g / (1 + np.exp(-g)) * np.where(np.arange(32) % 3, 1.0, -1.0) * 2.0 ** 100
    assert (g < -89).sum() > 20 and (np.abs(h) > 2.0 ** -109).all()
    # two exponentials within 2 steps each (4 half steps), their product twice that, four roundings, the third
    # plane's last step, and the down projection's exact power of two
    assert (np.abs(hidden_through(x, gate, up, 20, T, dev) * 2.0 ** -20 - h) <= 16 * 2.0 ** -24 * np.abs(h)).all()
