"""The plans of the MX4 and expert kernels (CPU only)."""
import pytest

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
