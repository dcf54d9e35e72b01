"""The MX4 and mixture-of-experts entry points refuse what they cannot do before anything reaches the
GPU, and their host-side sizes (CPU only)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import mx4_reference as ref
from decode_gemv_thinkbit_amd import qlinear as ql

FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation first
ODD = 0x10008


def message():
    return ql.lib().qlinear_last_error().decode()


def test_reference_quantiser_pins():
    """Hand-computed blocks: 6 sets the exponent 0; ties go to even codes; a value of 7 saturates."""
    x = np.zeros((1, 32))
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -7]
    codes, scales = ref.quantize(x)
    assert scales[0, 0] == 127 and list(scales[0, 1:]) == [0, 0, 0]
    assert list(codes[0, :5]) == [7 | 0 << 4, 2 | 2 << 4, 4 | 4 << 4, 6 | 6 << 4, 15]
    assert list(ref.values(codes, scales)[0, :9]) == [6, 0, 1, 1, 2, 2, 4, 4, -6]
    codes, scales = ref.quantize(np.full((1, 32), 2.0 ** -5))
    assert scales[0, 0] == 120 and codes[0, 0] == 0x66  # 4 * 2^-7


def test_limits_match_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "qlinear.h")).read()
    for name in ("EXPERTS", "TOPK", "TOKENS"):
        assert int(re.search(rf"#define QL_MOE_MAX_{name} (\d+)", src).group(1)) == getattr(ql, "MOE_MAX_" + name)


def test_scale_stride():
    L = ql.lib()
    for K, want in ((32, 4), (128, 4), (160, 8), (4096, 128), (2080, 68), (0, 0), (33, 0), (-32, 0), ((1 << 26) + 32, 0)):
        assert L.qlinear_mx4_scale_stride(K) == want, K


def test_tensor_refusals():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    t = ql.Mx4Tensor(u8(5, 80), u8(5, 8))
    assert (t.N, t.K, t.shape, t.nbytes) == (5, 160, (5, 160), 440)
    assert ql.Mx4Tensor(u8(3, 5, 16), u8(3, 5, 4)).shape == (3, 5, 32)
    with pytest.raises(AttributeError):  # its shape was checked
        t.codes = u8(9, 80)
    for codes, scales in ((u8(5, 80), u8(5, 5)), (u8(5, 80), u8(4, 8)), (u8(5, 24), u8(5, 4)), (u8(80), u8(8)),
                          (u8(0, 16), u8(0, 4)), (u8(80, 5).t(), u8(5, 8)), (u8(5, 16).float(), u8(5, 4)),
                          (u8(5, 16), u8(5, 4).to(torch.int8)), (u8(2, 2, 2, 16), u8(2, 2, 2, 4))):
        with pytest.raises(ValueError):
            ql.Mx4Tensor(codes, scales)


def test_host_tensors_are_refused():
    t = ql.Mx4Tensor(torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(16, 4, dtype=torch.uint8))
    s = ql.Mx4Tensor(torch.zeros(2, 16, 64, dtype=torch.uint8), torch.zeros(2, 16, 4, dtype=torch.uint8))
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    for call in (lambda: ql.mx4_quantize(x), lambda: ql.mx4_dequant(t), lambda: ql.mx4_gemv(x, t),
                 lambda: ql.mx4_gemm(t, t), lambda: ql.moe_route(torch.zeros(2, 8), 2),
                 lambda: ql.mx4_moe(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1), s, s, s)):
        with pytest.raises(ValueError):
            call()


def test_quantize_and_dequant_refusals():
    L = ql.lib()
    for N, K, ty, W, c, s in ((0, 32, 0, FAKE, FAKE, FAKE), (4, 0, 0, FAKE, FAKE, FAKE), (4, 48, 0, FAKE, FAKE, FAKE),
                              (4, 32, 3, FAKE, FAKE, FAKE), (4, 32, -1, FAKE, FAKE, FAKE), (4, 32, 0, None, FAKE, FAKE),
                              (4, 32, 0, FAKE, ODD, FAKE), (4, 32, 0, FAKE, FAKE, ODD),
                              (1 << 40, 32, 0, FAKE, FAKE, FAKE), (1, (1 << 26) + 32, 0, FAKE, FAKE, FAKE)):
        assert L.qlinear_mx4_quantize(N, K, ty, W, c, s, None) == 1 and message()
    for N, K, c, s, out in ((4, 33, FAKE, FAKE, FAKE), (-1, 32, FAKE, FAKE, FAKE), (4, 32, FAKE, FAKE, None),
                            (4, 32, FAKE, ODD, FAKE)):
        assert L.qlinear_mx4_dequant(N, K, c, s, 0, out, None) == 1 and message()


def test_product_refusals():
    L = ql.lib()
    for M, N, K, c, s, x, y in ((0, 16, 128, FAKE, FAKE, FAKE, FAKE), (17, 16, 128, FAKE, FAKE, FAKE, FAKE),
                                (1, 16, 100, FAKE, FAKE, FAKE, FAKE), (1, 0, 128, FAKE, FAKE, FAKE, FAKE),
                                (1, 1 << 26, 128, FAKE, FAKE, FAKE, FAKE), (1, 16, 128, ODD, FAKE, FAKE, FAKE),
                                (1, 16, 128, FAKE, None, FAKE, FAKE), (1, 16, 128, FAKE, FAKE, ODD, FAKE),
                                (1, 16, 128, FAKE, FAKE, FAKE, None)):
        assert L.qlinear_mx4_gemv(M, N, K, c, s, x, y, FAKE, 1 << 40, None) == 1 and message()
    assert L.qlinear_mx4_gemv(1, 16, (1 << 24) + 32, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == 1
    for M, N, K in ((0, 16, 128), (17, 16, 128), (1, 16, 100), (1, 0, 128)):
        assert L.qlinear_mx4_gemv_workspace_bytes(M, N, K) == 0
    for M, N, K, p in ((0, 16, 128, FAKE), (1 << 24, 16, 128, FAKE), (16, 16, 96 + 1, FAKE), (16, 1 << 26, 32, FAKE),
                       (16, 16, 128, ODD), (16, 16, 128, None)):
        assert L.qlinear_mx4_gemm(M, N, K, FAKE, FAKE, p, FAKE, FAKE, FAKE, 1 << 40, None) == 1 and message()


def test_route_refusals():
    L = ql.lib()
    for T, E, k, ty, p in ((0, 8, 2, 0, FAKE), (1 << 26, 8, 2, 0, FAKE), (4, 0, 1, 0, FAKE), (4, 1025, 2, 0, FAKE),
                           (4, 8, 0, 0, FAKE), (4, 8, 9, 0, FAKE), (4, 64, 17, 0, FAKE), (4, 8, 2, 5, FAKE),
                           (4, 8, 2, 0, ODD), (4, 8, 2, 0, None)):
        assert L.qlinear_moe_route(T, E, k, 1, ty, p, FAKE, FAKE, None) == 1 and message()


def test_moe_refusals():
    L = ql.lib()
    ok = dict(E=8, H=128, I=64, k=2, ids=FAKE, weights=FAKE, gate_codes=FAKE, gate_scales=FAKE, up_codes=FAKE,
              up_scales=FAKE, down_codes=FAKE, down_scales=FAKE)
    call = lambda T=4, x=FAKE, y=FAKE, ws=FAKE, size=1 << 30, **k: L.qlinear_mx4_moe(
        ctypes.byref(ql.ql_mx4_experts(**{**ok, **k})), T, x, y, ws, size, None)
    assert L.qlinear_mx4_moe(None, 4, FAKE, FAKE, FAKE, 1 << 30, None) == 1
    for bad in (dict(T=0), dict(T=65), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=64, k=17), dict(H=100),
                dict(I=33), dict(H=0), dict(I=-32), dict(H=(1 << 18) + 32), dict(x=None), dict(y=ODD), dict(ws=None),
                dict(ids=None), dict(weights=ODD), dict(down_scales=None), dict(up_codes=ODD), dict(size=16)):
        assert call(**bad) == 1 and message(), bad
    assert L.qlinear_mx4_moe_workspace_bytes(65, 2, 8, 128, 64) == 0
    assert L.qlinear_mx4_moe_workspace_bytes(4, 2, 8, 128, 64) > 0
