"""The feed-forward operators' C ABI on the host: every declared symbol is exported, bad
plans are refused before a device is touched; and the 64-bit formulas that the GPU tests
hold the kernels to agree with differences."""
import ctypes
import os
import re

import pytest
import torch

import all_gather_gemm_agmm_gb300 as agmm
import feedforward_ref as ref
from all_gather_gemm_agmm_gb300 import feedforward as ff

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "agmm_feedforward.h")
ARGS = {"layer_norm": ff._LAYER_NORM_ARGS, "layer_norm_grad": ff._LAYER_NORM_GRAD_ARGS, "gated": ff._GATED_ARGS,
        "gated_grad": ff._GATED_GRAD_ARGS, "linear": ff._LINEAR_ARGS, "linear_grad": ff._LINEAR_GRAD_ARGS}
F32, BF16, F16 = 1, 0, 2


@pytest.fixture(scope="module")
def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_matches_binding(agmm_lib, header):
    declared = sorted(set(re.findall(r"\b(agmm_[a-z_]+)\s*\(", header)))
    assert declared == sorted(ff.FEEDFORWARD_SYMBOLS)
    for name in declared:
        assert hasattr(agmm_lib, name), name
    assert int(re.search(r"AGMM_FEEDFORWARD_HEAD_BYTES (\d+)", header).group(1)) == ff.HEAD_BYTES
    for name, code in ff.ACTIVATIONS.items():
        assert re.search(r"AGMM_ACT_%s = %d" % ((name or "none").upper(), code), header)


@pytest.mark.parametrize("name", ARGS)
def test_argument_structs_are_64_bit_fields(header, name):
    body = re.search(r"typedef struct \{([^}]*)\} agmm_%s_args_t" % name, header).group(1)
    fields = 0
    for s in filter(str.strip, body.split(";")):
        assert "int64_t" in s or "*" in s, s
        for f in s.split(","):
            n = re.search(r"\[(\d+)\]", f)
            fields += int(n.group(1)) if n else 1
    assert ARGS[name].size == 8 * fields


def _plan(lib, name, desc):
    h = ctypes.c_void_p(1234)
    st = getattr(lib, f"agmm_{name}_plan")(ctypes.byref(desc) if desc is not None else None, ctypes.byref(h))
    return st, h.value


@pytest.mark.parametrize("desc", [(0, BF16, 1e-5), (4, BF16, 1e-5), (12, BF16, 1e-5), (-8, BF16, 1e-5), (16392, BF16, 1e-5),
                                  (64, F32, 1e-5), (64, 9, 1e-5), (64, BF16, -1.0), (64, F16, float("nan")), (64, F16, float("inf"))])
def test_layer_norm_plan_refusals(agmm_lib, desc):
    assert _plan(ff._library(), "layer_norm", ff._LayerNormDesc(*desc)) == (agmm.AGMM_ERR_INVALID_ARG, None)
    assert agmm_lib.agmm_last_error().decode()


# k, n, activation, rhs_transpose, dtype
@pytest.mark.parametrize("desc", [(0, 64, 2, 0, BF16), (64, 0, 2, 0, BF16), (60, 64, 2, 0, BF16), (64, 100, 2, 0, BF16),
                                  ((1 << 20) + 8, 64, 2, 0, BF16), (64, (1 << 20) + 8, 2, 0, BF16), (-64, 64, 2, 0, BF16),
                                  (64, 64, -1, 0, BF16), (64, 64, 5, 0, BF16), (64, 64, 2, 2, BF16), (64, 64, 2, 0, F32),
                                  (64, 64, 2, 0, 7)])
@pytest.mark.parametrize("name", ["gated", "linear"])
def test_product_plan_refusals(agmm_lib, name, desc):
    assert _plan(ff._library(), name, ff._ProductDesc(*desc)) == (agmm.AGMM_ERR_INVALID_ARG, None)


def test_gated_needs_an_activation(agmm_lib):
    assert _plan(ff._library(), "gated", ff._ProductDesc(64, 64, 0, 0, BF16)) == (agmm.AGMM_ERR_INVALID_ARG, None)


def test_null_calls(agmm_lib):
    lib = ff._library()
    for name in ("layer_norm", "gated", "linear"):
        assert _plan(lib, name, None) == (agmm.AGMM_ERR_INVALID_ARG, None)
        assert getattr(lib, f"agmm_{name}_plan")(None, None) == agmm.AGMM_ERR_INVALID_ARG
        for call in ("run", "backward"):
            assert getattr(lib, f"agmm_{name}_{call}")(None, b"", None) == agmm.AGMM_ERR_INVALID_ARG
        getattr(lib, f"agmm_{name}_destroy")(None)  # no-op
        assert getattr(lib, f"agmm_{name}_workspace_bytes")(None) == 0


@pytest.mark.parametrize("wide", [2**31, 2**32 + 64, -2**32 + 64])
def test_widths_past_32_bits(wide):
    """A plan's description has them as int: 2^32 + 64 is not a plan of 64."""
    for make in (lambda: agmm.LayerNormPlan(wide), lambda: agmm.GatedPlan(wide, 64), lambda: agmm.LinearPlan(64, wide)):
        with pytest.raises(ValueError, match="32-bit"):
            make()


def test_unknown_activation():
    with pytest.raises(ValueError, match="activation"):
        agmm.GatedPlan(64, 64, activation="swish")


# ------------------------------------------------------- the formulas against differences
def _difference(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


@pytest.mark.parametrize("kind", [None, "silu", "gelu", "gelu_tanh", "relu"])
def test_activation_slopes(kind):
    z = torch.linspace(-7, 7, 400, dtype=torch.float64)  # 0 is not among them
    d = _difference(lambda x: ref.act(x, kind)[0], z, torch.ones_like(z))
    assert float((d - ref.act(z, kind)[1]).abs().max()) < 1e-8


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("transpose", [False, True])
def test_gated_gradients(kind, transpose):
    g = torch.Generator().manual_seed(1)
    new = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    t, k, n = 5, 7, 6
    x, d = new(t, k), new(t, n)
    wg, wu = (new(n, k) if transpose else new(k, n) for _ in range(2))
    f = lambda x, wg, wu: (ref.gated(x, wg, wu, kind, transpose, torch.float32)["out"][0] * d).sum()  # noqa: E731
    gate, up = (ref.product(x, w, transpose)[0] for w in (wg, wu))
    got = ref.gated_grad(d, x, wg, wu, gate, up, kind, transpose, torch.float32, torch.float32)
    for name, y, call in (("dx", x, lambda y: f(y, wg, wu)), ("dw_gate", wg, lambda y: f(x, y, wu)), ("dw_up", wu, lambda y: f(x, wg, y))):
        v = new(*y.shape)
        assert abs(float(_difference(call, y, v) - (got[name][0] * v).sum())) < 1e-6


@pytest.mark.parametrize("kind", [None, "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("transpose", [False, True])
def test_linear_gradients(kind, transpose):
    g = torch.Generator().manual_seed(2)
    new = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    t, k, n = 5, 7, 6
    x, d, b, r = new(t, k), new(t, n), new(n), new(t, n)
    w = new(n, k) if transpose else new(k, n)
    f = lambda x, w, b: (ref.linear(x, w, b, r, kind, transpose, torch.float32)["out"][0] * d).sum()  # noqa: E731
    pre = ref.product(x, w, transpose)[0] + b
    got = ref.linear_grad(d, x, w, pre, kind, transpose, torch.float32, torch.float32)
    for name, y, call in (("dx", x, lambda y: f(y, w, b)), ("dw", w, lambda y: f(x, y, b)), ("d_bias", b, lambda y: f(x, w, y))):
        v = new(*y.shape)
        assert abs(float(_difference(call, y, v) - (got[name][0] * v).sum())) < 1e-6


def test_layer_norm_gradients():
    g = torch.Generator().manual_seed(3)
    new = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, d, add = new(6, 24), new(24), new(24), new(6, 24), new(6, 24)
    f = lambda x, w, b: (ref.norm(x, w, b, 1e-5, torch.float32)["out"][0] * d).sum()  # noqa: E731
    stats = ref.norm(x, w, b, 1e-5, torch.float32)
    got = ref.norm_grad(d, x, stats["mean"][0], stats["rstd"][0], w, add, torch.float32, torch.float32)
    v = new(6, 24)
    assert abs(float(_difference(lambda y: f(y, w, b), x, v) + (add * v).sum() - (got["dx"][0] * v).sum())) < 1e-6
    v = new(24)
    assert abs(float(_difference(lambda y: f(x, y, b), w, v) - (got["d_weight"][0] * v).sum())) < 1e-6
    assert abs(float(_difference(lambda y: f(x, w, y), b, v) - (got["d_bias"][0] * v).sum())) < 1e-6
