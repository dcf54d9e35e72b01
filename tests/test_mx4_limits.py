"""Limits and refusals of the MX4 and expert entry points at their borders (CPU only)."""

import pytest
import torch

from decode_gemv_thinkbit_amd import qlinear as ql

FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation first


def message():
    return ql.lib().qlinear_last_error().decode()


def test_route_grid_stays_below_two_to_the_32_threads():
    """Four tokens to a workgroup of 256 threads: from 2^26 - 3 tokens on a launch would have 2^32 threads."""
    for T in ((1 << 26) - 3, (1 << 26) - 2, (1 << 26) - 1):
        assert (T + 3) // 4 * 256 >= 1 << 32
        assert ql.lib().qlinear_moe_route(T, 8, 2, 1, 0, FAKE, FAKE, FAKE, None) == 1 and "2^26 - 4" in message()


def test_dequant_takes_only_mx4_tensors():
    codes = torch.zeros(4, 16, dtype=torch.uint8)
    for t in (codes, (codes, codes), None):
        with pytest.raises(ValueError, match="Mx4Tensor"):
            ql.mx4_dequant(t)
