"""The feed-forward products at the last number of tokens that one swapped tile holds, and the first that
it does not: 64 and 65 of one shard; shards that fill its 64 columns with their padding, and one row more."""
import pytest
import torch

from feedforward_ref import check, gated, gated_grad, linear, linear_grad

pytestmark = pytest.mark.gpu
# shards, rows: a shard's rows are padded to a multiple of 8
TOKENS = [(1, 63), (1, 64), (1, 65), (2, 32), (2, 33), (3, 16), (3, 17), (4, 13), (4, 17), (8, 8), (8, 9)]


@pytest.fixture(scope="module")
def agmm():
    import all_gather_gemm_agmm_gb300 as m
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    m.load_library()
    return m


def make(shards, rows, k, n, transpose, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
    shape = (n, k) if transpose else (k, n)
    return new, [new(rows, k) for _ in range(shards)], new(*shape, std=k ** -0.5), new(*shape, std=k ** -0.5), new(shards * rows, n)


def empty(dtype, *s):
    """Three rows more than are written."""
    return torch.full((s[0] + 3, *s[1:]), 7.0, dtype=dtype, device="cuda")


def held(buf, rows, want, name):
    check(buf[:rows], *want, name)
    assert bool((buf[rows:] == 7).all()), name


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shards, rows", TOKENS)
def test_gated(agmm, shards, rows, transpose):
    k, n, t = 520, 264, shards * rows
    dtype = torch.float16 if transpose else torch.bfloat16
    new, xs, wg, wu, d = make(shards, rows, k, n, transpose, dtype, 1)
    plan = agmm.GatedPlan(k, n, rhs_transpose=transpose, f16=transpose)
    ws = plan.new_workspace()
    got = {name: empty(dtype, t, n) for name in ("out", "gate", "up")}
    plan.run(xs, wg, wu, got["out"][:t], ws, gate=got["gate"][:t], up=got["up"][:t])
    want = gated(torch.cat(xs), wg, wu, "silu", transpose, dtype)
    for name, x in got.items():
        held(x, t, want[name], name)
    g, u = new(t, n), new(t, n)
    got = dict(d_gate=empty(dtype, t, n), d_up=empty(dtype, t, n), dx=empty(dtype, t, k))
    dw = [empty(dtype, *wg.shape) for _ in range(2)]
    s = wg.shape[0]
    plan.backward(d, xs, wg, wu, g, u, got["d_gate"][:t], got["d_up"][:t], ws, dx=got["dx"][:t], dw_gate=dw[0][:s], dw_up=dw[1][:s])
    plan.query_status(ws)
    want = gated_grad(d, torch.cat(xs), wg, wu, g, u, "silu", transpose, dtype, dtype)
    for name, x in got.items():
        held(x, t, want[name], name)
    held(dw[0], s, want["dw_gate"], "dw_gate")
    held(dw[1], s, want["dw_up"], "dw_up")


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shards, rows", TOKENS)
def test_linear(agmm, shards, rows, transpose):
    k, n, t = 264, 1032, shards * rows
    dtype = torch.bfloat16 if transpose else torch.float16
    new, xs, w, _, d = make(shards, rows, k, n, transpose, dtype, 2)
    bias, residual, pre = new(n), new(t, n), new(t, n)
    plan = agmm.LinearPlan(k, n, activation="relu", rhs_transpose=transpose, f16=not transpose)
    ws = plan.new_workspace()
    got = dict(out=empty(dtype, t, n), pre=empty(dtype, t, n))
    plan.run(xs, w, got["out"][:t], ws, bias=bias, residual=residual, pre=got["pre"][:t])
    want = linear(torch.cat(xs), w, bias, residual, "relu", transpose, dtype)
    for name, x in got.items():
        held(x, t, want[name], name)
    got = dict(d_pre=empty(dtype, t, n), dx=empty(dtype, t, k))
    s = w.shape[0]
    dw, db = empty(torch.float32, *w.shape), empty(torch.float32, n)
    plan.backward(d, xs, w, ws, pre=pre, d_pre=got["d_pre"][:t], dx=got["dx"][:t], dw=dw[:s], d_bias=db[:n])
    plan.query_status(ws)
    want = linear_grad(d, torch.cat(xs), w, pre, "relu", transpose, dtype, torch.float32)
    for name, x in got.items():
        held(x, t, want[name], name)
    held(dw, s, want["dw"], "dw")
    held(db, n, want["d_bias"], "d_bias")
