"""Loads straight into LDS are written in assembly blocks, where the compiler counts no wait states: the
device code compiled for gfx950 keeps them (CPU only).

- A load's scalar address is not written by a vector instruction (a lane read) in the five wait states
  before it, nor m0 by any instruction in the one before it.
- Where a block narrows the active lanes, all of them are active again right behind its last load.
- Every kernel with such loads waits for all of them before it ends: every path of the code from a load to
  the end passes a wait for a count of 0.
"""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from decode_gemv_thinkbit_amd import build as qb

SOURCES = ["ql_mx4.hip", "ql_mx4_gemm.hip", "ql_moe.hip"]


def device_asm(src):
    flags = [f for f in qb.FLAGS if f != "-fPIC"]
    r = subprocess.run([qb.HIPCC, *flags, "--offload-device-only", "-S", "-o", "-", os.path.join(qb.CSRC, src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


@pytest.fixture(scope="module")
def kernels():
    """{source: {kernel: [(instruction, operands)]}}; a label is an instruction without operands"""
    if not os.path.exists(qb.HIPCC):
        pytest.skip("hipcc not available")
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        texts = dict(zip(SOURCES, ex.map(device_asm, SOURCES)))
    out = {}
    for src, text in texts.items():
        for name, body in re.findall(r"^(_ZN2ql\w*kernel\w*):(.*?)\.Lfunc_end", text, re.M | re.S):
            lines = [line.split(";")[0].strip() for line in body.split("\n")]
            code = [line.replace(",", " ").split() for line in lines
                    if line and (not line.startswith(".") or line.startswith(".LBB"))]
            out.setdefault(src, {})[name] = [(c[0], c[1:]) for c in code]
    return out


def scalars(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m[1])} if m else set()


def states(op, operands):
    return int(operands[0], 0) + 1 if op == "s_nop" else 0 if op.startswith(".LBB") else 1


@pytest.mark.parametrize("src", SOURCES)
def test_wait_states_before_loads(kernels, src):
    seen = 0
    for name, code in kernels[src].items():
        for at, (op, operands) in enumerate(code):
            if not op.startswith("global_load_lds"):
                continue
            seen += 1
            used = scalars(operands[1]) if len(operands) > 1 else set()
            before = 0  # wait states between the instruction looked at and the load
            for o, r in reversed(code[max(0, at - 8):at]):
                if before < 5 and o.startswith("v_") and r:
                    assert not scalars(r[0]) & used, (name, o, r, operands, before)
                if before < 1 and r and r[0] == "m0":
                    raise AssertionError((name, "m0 written right before", operands))
                before += states(o, r)
    assert seen > 0


@pytest.mark.parametrize("src", SOURCES)
def test_all_lanes_return(kernels, src):
    for name, code in kernels[src].items():
        for at, (op, operands) in enumerate(code):
            if op.startswith("s_mov_b32") and operands[0] == "exec_hi":
                after = [c for c in code[at + 1:at + 9]]
                loads = [i for i, (o, _) in enumerate(after) if o.startswith("global_load_lds")]
                assert loads, name
                follow = after[loads[0] + 1]
                assert follow[0] == "s_mov_b64" and follow[1] == ["exec", "-1"] or \
                    follow[0] == "s_mov_b32" and follow[1][0] == "exec_lo", (name, follow)


@pytest.mark.parametrize("src", SOURCES)
def test_loads_end_before_the_kernel(kernels, src):
    for name, code in kernels[src].items():
        at_label = {op[:-1]: i for i, (op, _) in enumerate(code) if op.startswith(".LBB")}
        seen = set()
        todo = [i + 1 for i, (op, _) in enumerate(code) if op.startswith("global_load_lds")]
        while todo:
            i = todo.pop()
            if i in seen:
                continue
            seen.add(i)
            op, operands = code[i]
            assert op != "s_endpgm", name
            assert not op.startswith(("s_setpc", "s_swappc", "s_call")), name
            if op == "s_waitcnt" and "vmcnt(0)" in operands:
                continue
            if op.startswith(("s_branch", "s_cbranch")):
                todo.append(at_label[operands[0]])
            if op != "s_branch":
                todo.append(i + 1)
