"""The attention kernels' loads straight into LDS keep the rules that test_isa_lds_loads.py states, read from the
device code compiled for gfx950 (CPU only)."""
import pytest

import test_isa_lds_loads as rules

SOURCES = ["ql_attn_prompt.hip"]


@pytest.fixture(scope="module")
def kernels():
    with pytest.MonkeyPatch.context() as patch:
        patch.setattr(rules, "SOURCES", SOURCES)
        return rules.kernels.__wrapped__()


@pytest.mark.parametrize("src", SOURCES)
def test_wait_states_before_loads(kernels, src):
    rules.test_wait_states_before_loads(kernels, src)


@pytest.mark.parametrize("src", SOURCES)
def test_loads_end_before_the_kernel(kernels, src):
    rules.test_loads_end_before_the_kernel(kernels, src)


@pytest.mark.parametrize("src", SOURCES)
def test_all_lanes_return(kernels, src):
    assert any(op == "s_mov_b32" and operands[0] == "exec_hi" for code in kernels[src].values() for op, operands in code)
    rules.test_all_lanes_return(kernels, src)
