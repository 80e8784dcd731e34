"""Feed-forward operators over memory and rows that 32 bits do not count: rows 2 MiB apart (8 GiB to a
matrix) give the bits that rows next to one another give, and millions of tokens the formulas' values."""
import pytest
import torch

from feedforward_ref import check, gated, linear, linear_grad, norm, norm_grad

pytestmark = pytest.mark.gpu
STRIDE, ROWS = 1 << 20, 4101  # values from one row to the next: the last starts behind 2^32 bytes


@pytest.fixture(scope="module")
def agmm():
    import all_gather_gemm_agmm_gb300 as m
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def far(x=None, rows=ROWS, columns=0, dtype=torch.bfloat16):
    """x, or a matrix of sevens, with its rows far apart."""
    rows, columns = (rows, columns) if x is None else x.shape
    out = torch.empty(rows * STRIDE, dtype=dtype if x is None else x.dtype, device="cuda").view(rows, STRIDE)[:, :columns]
    return out.fill_(7) if x is None else out.copy_(x)


def new(g, *s, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(s, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("tokens, n", [(ROWS, 72), (40, 4104)])
def test_linear_rows_far_apart(agmm, tokens, n):
    g = torch.Generator(device="cuda").manual_seed(1)
    k = 136
    x, w, bias, r, d = new(g, tokens, k), new(g, n, k, std=0.1), new(g, n), new(g, tokens, n), new(g, tokens, n)
    plan = agmm.LinearPlan(k, n, activation="silu", rhs_transpose=True)
    ws = plan.new_workspace()
    near = [torch.empty_like(t) for t in (d, d, d, x, w)]
    apart = [far(rows=t.shape[0], columns=t.shape[1]) for t in near]
    db = torch.empty(2, n, dtype=torch.bfloat16, device="cuda")
    for i, (out, pre, d_pre, dx, dw) in enumerate((near, apart)):
        put = far if i else (lambda t: t)
        xi, wi = put(x), put(w)
        plan.run(xi, wi, out, ws, bias=bias, residual=put(r), pre=pre)
        plan.backward(put(d), xi, wi, ws, pre=pre, d_pre=d_pre, dx=dx, dw=dw, d_bias=db[i])
        plan.query_status(ws)
    for a, b in zip(near, apart):
        assert torch.equal(a, b)
    assert torch.equal(db[0], db[1])
    check(near[0], *linear(x, w, bias, r, "silu", True, torch.bfloat16)["out"], "out")


def test_gated_rows_far_apart(agmm):
    g = torch.Generator(device="cuda").manual_seed(2)
    k, n = 72, 136
    x, wg, wu, d = new(g, ROWS, k), new(g, k, n, std=0.1), new(g, k, n, std=0.1), new(g, ROWS, n)
    plan = agmm.GatedPlan(k, n, "gelu")
    ws = plan.new_workspace()
    near = [torch.empty_like(t) for t in (d, d, d, x)]
    apart = [far(rows=ROWS, columns=t.shape[1]) for t in near]
    dw = torch.empty(4, k, n, device="cuda")
    for i, (out, gate, up, dx) in enumerate((near, apart)):
        xi = far(x) if i else x
        plan.run(xi, wg, wu, out, ws, gate=gate, up=up)
        keep = gate.clone(), up.clone()
        plan.backward(far(d) if i else d, xi, wg, wu, gate, up, gate, up, ws, dx=dx, dw_gate=dw[2 * i], dw_up=dw[2 * i + 1])
        plan.query_status(ws)
    for a, b in zip(near, apart):
        assert torch.equal(a, b)
    assert torch.equal(dw[:2], dw[2:])
    want = gated(x, wg, wu, "gelu", False, torch.bfloat16)
    for name, got in zip(("out", "gate", "up"), (near[0], *keep)):
        check(got, *want[name], name)


@pytest.mark.parametrize("rows, columns", [(ROWS, 264), (ROWS, 1032), (ROWS, 8200)])
def test_layer_norm_rows_far_apart(agmm, rows, columns):
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w, b, d, add = new(g, rows, columns), new(g, columns), new(g, columns), new(g, rows, columns), new(g, rows, columns)
    plan = agmm.LayerNormPlan(columns)
    ws = plan.new_workspace()
    results = []
    for put in (lambda t: t, far):
        xi, out, dx = put(x), put(torch.empty_like(x)), put(torch.empty_like(x))
        mean, rstd, dw, db = (torch.empty(m, device="cuda") for m in (rows, rows, columns, columns))
        plan.run(xi, out, weight=w, bias=b, mean=mean, rstd=rstd)
        plan.backward(put(d), xi, mean, rstd, dx, ws, weight=w, add=put(add), d_weight=dw, d_bias=db)
        results.append((out, mean, rstd, dx, dw, db))
    for p, q in zip(*results):
        assert torch.equal(p, q)
    check(results[0][0], *norm(x, w, b, 1e-5, torch.bfloat16)["out"], "out")


def test_millions_of_rows(agmm):
    """2^22 + 3 tokens: tile numbers and a sum of 65537 k blocks."""
    g = torch.Generator(device="cuda").manual_seed(4)
    t, k, n = (1 << 22) + 3, 8, 16
    x, w, bias, d = new(g, t, k), new(g, k, n), new(g, n), new(g, t, n)
    plan = agmm.LinearPlan(k, n, activation="relu")
    ws = plan.new_workspace()
    out, pre, d_pre, dx, dw, db = (torch.empty_like(v) for v in (d, d, d, x, w, bias))
    plan.run(x, w, out, ws, bias=bias, pre=pre)
    plan.backward(d, x, w, ws, pre=pre, d_pre=d_pre, dx=dx, dw=dw, d_bias=db)
    plan.query_status(ws)
    check(out, *linear(x, w, bias, None, "relu", False, torch.bfloat16)["out"], "out")
    want = linear_grad(d, x, w, pre, "relu", False, torch.bfloat16, torch.bfloat16)
    for name, got in dict(d_pre=d_pre, dx=dx, dw=dw, d_bias=db).items():
        check(got, *want[name], name)


def test_millions_of_norms(agmm):
    g = torch.Generator(device="cuda").manual_seed(5)
    rows, columns = (1 << 22) + 3, 16
    x, w, b, d = new(g, rows, columns), new(g, columns), new(g, columns), new(g, rows, columns)
    out, mean, rstd = agmm.layer_norm(x, w, b, return_stats=True)
    check(out, *norm(x, w, b, 1e-5, torch.bfloat16)["out"], "out")
    dx, dw, db = agmm.layer_norm_backward(d, x, mean, rstd, w, f32_grads=True)
    want = norm_grad(d, x, mean, rstd, w, None, torch.bfloat16, torch.float32)
    for name, got in dict(dx=dx, d_weight=dw, d_bias=db).items():
        check(got, *want[name], name)
