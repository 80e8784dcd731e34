"""The attention operators' C ABI on the host: every declared symbol is
exported, and bad plans are refused before a device is touched."""
import ctypes
import os
import re

import pytest

import all_gather_gemm_agmm_gb300 as agmm
from all_gather_gemm_agmm_gb300 import attention

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "agmm_attention.h")


@pytest.fixture(scope="module")
def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_matches_binding(agmm_lib, header):
    declared = sorted(set(re.findall(r"\b(agmm_[a-z_]+)\s*\(", header)))
    assert declared == sorted(attention.ATTENTION_SYMBOLS)
    for name in declared:
        assert hasattr(agmm_lib, name), name


@pytest.mark.parametrize("name,packed", [("norm_rope", attention._NORM_ROPE_ARGS), ("prompt", attention._PROMPT_ARGS),
                                         ("tree", attention._TREE_ARGS)])
def test_argument_structs_are_64_bit_fields(header, name, packed):
    body = re.search(r"typedef struct \{([^}]*)\} agmm_%s_args_t" % name, header).group(1)
    fields = [f for s in body.split(";") if s.strip() for f in s.split(",")]
    assert all("int64_t" in s or "*" in s for s in body.split(";") if s.strip())
    assert packed.size == 8 * len(fields)


def _plan(lib, name, desc):
    h = ctypes.c_void_p(1234)
    st = getattr(lib, f"agmm_{name}_plan")(ctypes.byref(desc) if desc is not None else None, ctypes.byref(h))
    return st, h.value


@pytest.mark.parametrize("args", [(0, 1, 64, 1, 0), (4, 0, 64, 1, 0), (4, 3, 64, 1, 0), (4, 2, 64, 1, 1), (4, 2, 64, 1, 9)])
def test_prompt_plan_refusals(agmm_lib, args):
    lib = attention._library()
    assert _plan(lib, "prompt", attention._PromptDesc(*args, 1.0)) == (agmm.AGMM_ERR_INVALID_ARG, None)


def test_unsupported_and_not_finite(agmm_lib):
    lib = attention._library()
    assert _plan(lib, "prompt", attention._PromptDesc(4, 2, 96, 1, 0, 1.0)) == (agmm.AGMM_ERR_UNSUPPORTED, None)
    assert _plan(lib, "prompt", attention._PromptDesc(4, 2, 64, 1, 0, float("nan"))) == (agmm.AGMM_ERR_INVALID_ARG, None)
    assert _plan(lib, "tree", attention._TreeDesc(4, 2, 64, 24, 1, 0, 1.0)) == (agmm.AGMM_ERR_UNSUPPORTED, None)
    assert _plan(lib, "tree", attention._TreeDesc(4, 2, 64, 4, 1, 0, 1.0)) == (agmm.AGMM_ERR_UNSUPPORTED, None)
    assert _plan(lib, "tree", attention._TreeDesc(4, 2, 64, 16, 0, 0, 1.0)) == (agmm.AGMM_ERR_INVALID_ARG, None)
    assert _plan(lib, "tree", attention._TreeDesc(300, 1, 64, 16, 1, 0, 1.0)) == (agmm.AGMM_ERR_UNSUPPORTED, None)
    for name in ("norm_rope", "prompt", "tree"):
        assert _plan(lib, name, None) == (agmm.AGMM_ERR_INVALID_ARG, None)
        assert getattr(lib, f"agmm_{name}_run")(None, b"", None) == agmm.AGMM_ERR_INVALID_ARG
        getattr(lib, f"agmm_{name}_destroy")(None)  # no-op
    assert lib.agmm_tree_workspace_bytes(None) == 0


def test_rotary_axes():
    assert agmm.rotary_axes((2, 3)) == [0, 0, 1, 1, 1]
    assert agmm.rotary_axes((4, 2, 2), interleaved=True) == [0, 1, 2, 0, 1, 2, 0, 0]


def test_tree_mask():
    m = agmm.tree_mask([[-1, 0, 0, 1], [-1]], device="cpu")
    assert m.tolist() == [[1], [3], [5], [11], [1]]
    chain = agmm.tree_mask([list(range(-1, 69))], device="cpu")
    assert chain.shape == (70, 2) and chain[69].tolist() == [-1, 63] and chain[63].tolist() == [-1, 0]
    with pytest.raises(ValueError):
        agmm.tree_mask([[0]], device="cpu")
    with pytest.raises(ValueError):
        agmm.tree_mask([list(range(-1, 69))], words=1, device="cpu")
