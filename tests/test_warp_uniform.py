"""Code that a whole warp runs takes its turns by answers that are the same for all lanes.

A lane's own look at a barrier is not: PTX promises neither that the lanes of a warp look at the same
moment, nor that they get one answer.  A branch on it in front of a shuffle or a vote over the full warp
would leave lanes in different ones, for good.  So such an answer is voted on, and the result of a wait
comes from one lane, before a branch.  (A warp that comes apart cannot be made to on a GPU at will, and
would hang it: this reads the source.)"""
import os
import re

import pytest

PACKAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "all_gather_gemm_agmm_gb300")
KERNELS = ["csrc/agmm_fused_kernel.cuh", "csrc_feedforward/ff_gemm.cuh"]


def code(name):
    text = open(os.path.join(PACKAGE, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def conditions(text):
    """What stands in the parentheses of every if and while."""
    for m in re.finditer(r"\b(?:if|while)\s*(?:constexpr\s*)?\(", text):
        depth, end = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[end], 0)
            end += 1
        yield text[m.end():end - 1]


@pytest.mark.parametrize("kernel", KERNELS)
def test_looks_ahead_are_voted_on(kernel):
    text = code(kernel)
    names = set(re.findall(r"\b(\w+)\s*=[^;=]*\bmbar_test_wait\(", text))
    assert names, "no look ahead: this test has nothing to hold"
    asked = 0
    for c in conditions(text):
        for name in names:
            if re.search(r"\b%s\b" % name, c):
                assert c.replace(" ", "") == "!__all_sync(0xffffffffu,%s)" % name, c
                asked += 1
    assert asked == len(names) == len(re.findall(r"\bmbar_test_wait\(", text.split("__global__")[-1]))


@pytest.mark.parametrize("kernel", KERNELS)
def test_results_of_waits_come_from_one_lane(kernel):
    """In the roles' loops: `res = wait_phase(...)` of all lanes, or of lane 0, then one shuffle."""
    body = code(kernel).split("__global__")[-1]
    waits = re.findall(r"\bres = wait_phase(?:<\w+>)?\([^;]*;\s*([^;]*);", body)
    assert waits
    for following in waits:
        assert following == "res = __shfl_sync(0xffffffffu, res, 0)", following


@pytest.mark.parametrize("kernel", KERNELS)
def test_no_collective_behind_a_lane_s_own_flag(kernel):
    """Another warp may raise the abort flag between two lanes' reads of it: what the warp does together
    (loads of tensor memory, elections) stands behind a vote on it."""
    body = code(kernel).split("__global__")[-1]
    for c in conditions(body):
        if "*abort_flag" in c:
            assert "elect_one" not in c or "__any_sync(0xffffffffu, *abort_flag)" in c, c
    for m in re.finditer(r"if \(!?\*abort_flag\) \{", body):
        depth, end = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(body[end], 0)
            end += 1
        assert not re.search(r"tmem_ld|elect_one|_sync\(", body[m.end():end]), body[m.start():m.start() + 200]
