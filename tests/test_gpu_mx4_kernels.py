"""Every compiled form of the MX4 decode GEMV and GEMM, bit for bit: random codes and scales whose sums are exact in
fp32, against the fp64 product of the same values."""
import pytest
import torch

import mx4_cases as cases
from decode_gemv_thinkbit_amd import qlinear as ql

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ql.lib()
    return torch.device("cuda:0")


def seeded(M, N, K, dev):
    return torch.Generator(device=dev).manual_seed(M * 1000003 + N * 1009 + K)


@pytest.mark.parametrize("M,N,K", cases.GEMV)
def test_gemv_is_exact(dev, M, N, K):
    g = seeded(M, N, K, dev)
    w = cases.integers((N,), K, g, dev)
    x = torch.randint(-4, 5, (M, K), generator=g, device=dev).bfloat16()
    want = cases.exact_product(x.double(), cases.values(w), 0.25)
    y = ql.mx4_gemv(x, w)
    assert torch.equal(y.double(), want), (int((y.double() != want).sum()), y.numel())


@pytest.mark.parametrize("M,N,K", cases.GEMM)
def test_gemm_is_exact(dev, M, N, K):
    g = seeded(M, N, K, dev)
    w, x = cases.integers((N,), K, g, dev), cases.integers((M,), K, g, dev)
    want = cases.exact_product(cases.values(x), cases.values(w), 0.0625)
    y = ql.mx4_gemm(x, w)
    assert torch.equal(y.double(), want), (int((y.double() != want).sum()), y.numel())
