"""The plans of the MX4 and expert kernels (CPU only)."""
import itertools

import pytest

import mx4_cases as cases
import mx4_plans as plans


@pytest.mark.parametrize("T,k,E,H,I,gate,down", [
    (9, 8, 60, 2048, 1024, 11, 12),    # about 2780 tasks of each kernel: one round of 11 x 256 and 12 x 256 waves
    (24, 8, 128, 2048, 768, 11, 10),   # two rounds of 11, three of 9
    (12, 6, 128, 2080, 736, 11, 10),
    (20, 4, 32, 2048, 1408, 11, 10),   # few tasks in the second kernel: one round either way
    (16, 8, 60, 2048, 1024, 9, 10),    # two rounds either way
    (24, 6, 128, 2080, 736, 9, 10),
    (33, 4, 16, 2048, 2048, 9, 10),    # one round either way
    (8, 8, 60, 2048, 1024, 11, 12),    # up to 64 pairs
    (32, 8, 64, 4096, 1536, 9, 10),    # three rounds either way
    (64, 8, 128, 4096, 1536, 9, 8),    # tasks of 64 rows in the second kernel
])
def test_waves_follow_the_tasks(T, k, E, H, I, gate, down):
    p = plans.moe_plan(T, k, E, H, I)
    assert (p.gate_waves, p.down_waves) == (gate, down)


def test_gemv_cases_run_every_kernel():
    got = {plans.gemv(*c) for c in cases.GEMV}
    assert got == set(itertools.product((1, 2, 4), (1, 2, 4, 8), (False, True), (False, True)))


def test_gemm_cases_run_every_kernel():
    got = {plans.gemm(*c) for c in cases.GEMM}
    assert got == (set(itertools.product(("skinny",), (1, 2, 4), (1, 2, 4), (False, True), (False, True)))
                   | set(itertools.product(("tile",), ("64x64", "64x128", "128x128", "256x256"), (False, True))))
    for tile in ("64x64", "64x128", "128x128", "256x256"):  # chunks past whole quads of scales; more than one quad
        Ks = [K for M, N, K in cases.GEMM if plans.gemm(M, N, K)[:2] == ("tile", tile)]
        assert {(K + 127) // 128 % 4 for K in Ks} == {0, 1, 2, 3} and max(Ks) > 1024


def test_moe_cases_run_every_kernel():
    got = [plans.moe(*c) for c in cases.MOE]
    assert {g for g, _ in got} == {(*kind, tail) for tail in (False, True) for kind in (
        (1, 4, True, True), (2, 4, True, True), (1, 16, False, True), (8, 11, False, True), (8, 11, False, False),
        (8, 9, False, False))}
    downs = {d for _, d in got}
    ones = {d for d in downs if d[0] == "one"}
    assert downs - ones == {(*kind, tail) for tail in (False, True) for kind in (
        *(("few", 12, split) for split in (1, 2, 3, 4, 6, 12)), ("many", 10, 1), ("many", 12, 1), ("wide", 8, 1))}
    assert {d[3] for d in ones} == {False, True} and {1, 2, 3, 5, 16} <= {d[2] for d in ones}
