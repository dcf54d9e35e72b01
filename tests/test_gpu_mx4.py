"""Microscaled 4-bit floats on the GPU against plain 64-bit references: quantisation and its inverse
(bit-exact), the decode GEMV and the MX4 x MX4 GEMM (within the fp32 summation bound)."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from decode_gemv_thinkbit_amd import qlinear as ql

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ql.lib()
    return torch.device("cuda:0")


def activations(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(M, K, generator=g).to(torch.bfloat16)


def check(y, want, bound, what):
    y = y.cpu().numpy().astype(np.float64)
    bad = np.abs(y - want) > bound + 1e-300
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(y - want) / (bound + 1e-300)).max()))


# ---------------------------------------------------------------- quantise and back
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (2, 128), (17, 160), (70, 640), (2, 5, 64)])
def test_quantize_matches_definition(dev, kind, shape):
    g = torch.Generator().manual_seed(sum(shape))
    W = (torch.randn(*shape, generator=g) * torch.exp2(torch.randint(-12, 8, shape, generator=g).float())).to(TYPES[kind])
    t = ql.mx4_quantize(W.to(dev))
    codes, scales = ref.quantize(W.double().numpy())
    assert np.array_equal(t.codes.cpu().numpy(), codes)
    assert np.array_equal(t.scales.cpu().numpy(), scales)
    assert np.array_equal(ql.mx4_dequant(t).cpu().numpy().astype(np.float64), ref.values(codes, scales))


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_quantize_special_blocks(dev, kind):
    """Ties, zeros, saturation, the type's extremes, subnormals, infinities and NaN."""
    ty = TYPES[kind]
    info = torch.finfo(ty)
    tiny = 2.0 ** -24 if kind == "fp16" else 2.0 ** -133
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.5, 4.0]
    rows = [
        ties + [-v for v in ties] + [0.0] * 12,
        [0.0] * 32,
        [-0.0] * 16 + [0.0] * 16,
        [info.max] + [info.max / 3] * 30 + [-info.max],
        [tiny] * 31 + [-tiny],
        [info.tiny * v / 8 for v in range(32)],
        [2.0 ** -14 * v for v in range(32)],
        [1.0] * 31 + [float("inf")],
        [float("-inf")] + [0.0] * 31,
        [float("nan")] + [1.0] * 31,
        [1e-3] * 31 + [1.0],
    ]
    W = torch.tensor(rows, dtype=torch.float64).to(ty)
    t = ql.mx4_quantize(W.to(dev))
    codes, scales = ref.quantize(W.double().numpy())
    assert np.array_equal(t.scales.cpu().numpy(), scales)
    got = t.codes.cpu().numpy()
    for i in range(len(rows)):
        assert np.array_equal(got[i], codes[i]), (i, got[i], codes[i])
    back = ql.mx4_dequant(t).cpu().numpy()
    assert np.isnan(back[7:10]).all() and np.isfinite(back[:7]).all()


def test_dequant_every_code_and_scale(dev):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).view(256, 16, 16)  # 16 blocks hold every byte
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1, 1).repeat(1, 16, 4)
    t = ql.Mx4Tensor(codes.contiguous().to(dev), scales.contiguous().to(dev))
    want = ref.host(t)
    with np.errstate(over="ignore"):
        want32 = want.astype(np.float32)
    got = ql.mx4_dequant(t).cpu().numpy()
    assert np.array_equal(got, want32, equal_nan=True)
    assert np.array_equal(np.signbit(got[:255]), np.signbit(want32[:255]))
    got16 = ql.mx4_dequant(t, out_bf16=True).cpu().float().numpy()
    assert np.array_equal(got16, want32, equal_nan=True)


def test_quantize_into_given_tensors(dev):
    W = torch.randn(9, 224, device=dev)
    a = ql.mx4_quantize(W)
    b = ql.Mx4Tensor(torch.full_like(a.codes, 0xEE), torch.full_like(a.scales, 0xEE))
    assert ql.mx4_quantize(W, out=b) is b
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    assert (b.scales[:, 7:] == 0).all()  # the padding of 7 blocks to 8
    out = torch.empty(9, 224, device=dev)
    assert ql.mx4_dequant(a, out=out) is out and torch.equal(out, ql.mx4_dequant(b))


# ---------------------------------------------------------------- decode GEMV
GEMV = [(1, 1, 32), (1, 16, 128), (1, 17, 96), (2, 15, 160), (3, 100, 1056), (4, 64, 4096), (5, 1000, 2080),
        (7, 33, 640), (8, 272, 512), (9, 48, 12288), (15, 31, 224), (16, 16, 128), (16, 129, 2048), (16, 1, 17408),
        (1, 4096, 2048), (12, 2053, 736)]


@pytest.mark.parametrize("M,N,K", GEMV)
def test_gemv(dev, M, N, K):
    w = ref.random_mx4((N, K), 7 * N + K, dev)
    x = activations(M, K, M + K)
    y = ql.mx4_gemv(x.to(dev), w)
    assert y.shape == (M, N)
    want, bound = ref.product(x.double().numpy(), ref.host(w))
    check(y, want, bound, (M, N, K))
    assert torch.equal(y, ql.mx4_gemv(x.to(dev), w))  # deterministic


def test_gemv_single_vector_and_guarded_output(dev):
    """A 1-D x, and an output inside a larger buffer: nothing beside it is written."""
    N, K = 37, 288
    w = ref.random_mx4((N, K), 3, dev)
    x = activations(1, K, 4).to(dev)
    buf = torch.full((64 + 3 * N + 64,), 7.0, device=dev)
    for M in (1, 3):
        buf.fill_(7.0)
        out = buf[64:64 + M * N].view(M, N)
        ql.mx4_gemv(x.view(-1) if M == 1 else x.expand(M, K).contiguous(), w, out=out)
        assert (buf[:64] == 7).all() and (buf[64 + M * N:] == 7).all()
        assert torch.equal(out, ql.mx4_gemv(x, w).expand(M, N))


@pytest.mark.parametrize("M", [1, 16])
def test_gemv_extreme_scales(dev, M):
    """Scale bytes 0 (products of subnormal weights) and large ones; exact sums, so bit-exact."""
    N, K = 20, 64
    codes = torch.full((N, K // 2), 0x21, dtype=torch.uint8)  # 0.5 and 1.0
    scales = torch.zeros((N, 4), dtype=torch.uint8)
    scales[:, 0] = torch.arange(N) * 12  # 2^-127 .. 2^101
    scales[:, 1] = scales[:, 0]
    x = torch.full((M, K), 2.0 ** 20, dtype=torch.bfloat16)
    y = ql.mx4_gemv(x.to(dev), ql.Mx4Tensor(codes.to(dev), scales.to(dev))).cpu().double()
    want = 48.0 * 2.0 ** 20 * torch.exp2(torch.arange(N).double() * 12 - 127)
    assert torch.equal(y, want.expand(M, N))


def test_nan_scale_stays_in_its_row(dev):
    N, K = 40, 256
    w = ref.random_mx4((N, K), 5, dev)
    w.scales[17, 3] = 255
    x = activations(16, K, 6).to(dev)
    xq = ql.mx4_quantize(x)
    for y in (ql.mx4_gemv(x, w), ql.mx4_gemm(xq, w)):
        bad = torch.isnan(y)
        assert bad[:, 17].all() and bad.sum() == 16
    xq.scales[5, 2] = 255
    bad = torch.isnan(ql.mx4_gemm(xq, w))
    assert bad[5].all() and bad[:, 17].all() and bad.sum() == N + 16 - 1


def test_scale_padding_is_ignored(dev):
    """Bytes past K/32 in a row of scales change nothing."""
    N, K = 50, 160
    w = ref.random_mx4((N, K), 8, dev)
    x = activations(9, K, 9).to(dev)
    xq = ql.mx4_quantize(x)
    before = ql.mx4_gemv(x, w), ql.mx4_gemm(xq, w), ql.mx4_dequant(w)
    w.scales[:, 5:] = 255
    xq.scales[:, 5:] = 255
    after = ql.mx4_gemv(x, w), ql.mx4_gemm(xq, w), ql.mx4_dequant(w)
    for a, b in zip(before, after):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- GEMM
GEMM = [(1, 1, 32), (1, 130, 96), (2, 64, 128), (16, 16, 160), (17, 129, 256), (31, 300, 1056), (33, 5120, 640),
        (64, 65, 4096), (65, 1000, 224), (128, 256, 512), (129, 127, 2048), (200, 257, 736), (257, 513, 384),
        (512, 512, 1024), (300, 1100, 17408), (1, 4096, 4096), (700, 96, 64)]


@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm(dev, M, N, K):
    w = ref.random_mx4((N, K), 7 * N + K, dev)
    x = ref.random_mx4((M, K), M + K, dev, 118, 132)
    y = ql.mx4_gemm(x, w)
    assert y.shape == (M, N)
    want, bound = ref.product(ref.host(x), ref.host(w))
    check(y, want, bound, (M, N, K))
    assert torch.equal(y, ql.mx4_gemm(x, w))  # deterministic


@pytest.mark.parametrize("M,N,K", [(3, 70, 288), (150, 140, 416)])
def test_gemm_one_hot_is_exact(dev, M, N, K):
    """x rows with a single 1.0: every output is one weight, bit for bit, at every input position."""
    w = ref.random_mx4((N, K), 11, dev, 0, 254)
    want = ref.host(w).astype(np.float32)
    for k0 in range(0, K, M):
        x = torch.zeros(M, K)
        for m in range(M):
            x[m, (k0 + m) % K] = 1.0
        y = ql.mx4_gemm(ql.mx4_quantize(x.to(dev)), w).cpu().numpy()
        for m in range(M):
            assert np.array_equal(y[m], want[:, (k0 + m) % K]), (k0, m)


def test_gemm_guarded_output(dev):
    M, N, K = 131, 70, 192
    w, x = ref.random_mx4((N, K), 1, dev), ref.random_mx4((M, K), 2, dev)
    buf = torch.full((64 + M * N + 64,), 7.0, device=dev)
    out = buf[64:64 + M * N].view(M, N)
    ql.mx4_gemm(x, w, out=out)
    assert (buf[:64] == 7).all() and (buf[64 + M * N:] == 7).all()
    assert torch.equal(out, ql.mx4_gemm(x, w))


# ---------------------------------------------------------------- beyond 32-bit offsets
def test_products_beyond_four_gigabytes(dev):
    """Rows whose codes lie beyond 4 GB, and outputs beyond 2^31 elements; exact sums (multiples of 0.5 far
    below 2^24), so equal to the last rows alone."""
    N, K, tail = 2200001, 4096, 130
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device=dev)
    codes[-tail:] = torch.randint(0, 256, (tail, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device=dev)
    w, last = ql.Mx4Tensor(codes, scales), ql.Mx4Tensor(codes[-tail:].clone(), scales[-tail:].clone())
    for M in (1, 11):
        x = torch.randint(-2, 3, (M, K), device=dev).bfloat16()
        assert torch.equal(ql.mx4_gemv(x, w)[:, -tail:], ql.mx4_gemv(x, last))
    for M in (40, 1000):
        x = ql.mx4_quantize(torch.randint(-4, 5, (M, K), device=dev).float())
        y = ql.mx4_gemm(x, w)
        assert M < 1000 or y.numel() > 1 << 31
        assert torch.equal(y[:, -tail:], ql.mx4_gemm(x, last)) and (y[:, :1000] == 0).all()
        del y


def test_quantize_beyond_two_billion(dev):
    N, K, tail = 1050000, 2080, 37
    W = torch.zeros(N, K, dtype=torch.bfloat16, device=dev)
    assert W.numel() > 1 << 31
    W[-tail:] = torch.randn(tail, K, device=dev)
    t, last = ql.mx4_quantize(W), ql.mx4_quantize(W[-tail:].clone())
    assert torch.equal(t.codes[-tail:], last.codes) and torch.equal(t.scales[-tail:], last.scales)
    assert (t.codes[:5] == 0).all() and (t.scales[:5] == 0).all()
    out = ql.mx4_dequant(t, out_bf16=True)
    assert torch.equal(out[-tail:], ql.mx4_dequant(last, out_bf16=True))
