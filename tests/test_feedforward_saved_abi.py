"""Refusals of the calls that set what a plan saves, on the host."""
import all_gather_gemm_agmm_gb300 as agmm
from all_gather_gemm_agmm_gb300 import feedforward as ff


def test_save_float_without_a_plan(agmm_lib):
    lib = ff._library()
    for name in ("gated", "linear"):
        assert getattr(lib, f"agmm_{name}_save_float")(None, 1) == agmm.AGMM_ERR_INVALID_ARG
        assert agmm_lib.agmm_last_error().decode()
