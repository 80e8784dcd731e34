"""The product with bias, activation and residual and its backward pass against the
64-bit formulas."""
import pytest
import torch

from feedforward_ref import check, linear, linear_grad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def agmm():
    import all_gather_gemm_agmm_gb300 as m
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    m.load_library()
    return m


def make(shards, rows, k, n, transpose, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
    xs = [new(rows, k) for _ in range(shards)]
    return (xs, new(*((n, k) if transpose else (k, n)), std=k ** -0.5), new(n), new(shards * rows, n), new(shards * rows, n))


# shards, rows, k, n, [n, k], fp16, activation, bias, residual
FORWARD = [
    (1, 1, 64, 128, True, False, None, False, False),
    (1, 1, 7168, 1024, True, False, None, False, True),   # cut along k, one token
    (1, 1, 8, 8, False, True, "gelu", True, True),
    (1, 9, 200, 136, False, False, "gelu_tanh", True, False),
    (2, 33, 1288, 520, True, True, "relu", True, True),
    (1, 128, 512, 384, False, True, "silu", False, True),
    (1, 129, 512, 384, True, False, None, True, True),
    (8, 16, 1024, 264, False, False, "gelu", True, True),
    (8, 17, 320, 200, True, False, None, False, True),
    (7, 100, 256, 384, False, True, "silu", True, False),
    (1, 1000, 136, 1000, False, False, "gelu", True, True),
    (1, 300, 4096, 512, True, False, None, True, True),   # few row tiles, cut along k
    (1, 2500, 512, 2304, True, True, "relu", True, True),
]


def ids(cases):
    return ["x".join(str(int(v) if isinstance(v, bool) else v) for v in c) for c in cases]


@pytest.mark.parametrize("case", FORWARD, ids=ids(FORWARD))
def test_forward(agmm, case):
    shards, rows, k, n, transpose, f16, kind, has_bias, has_residual = case
    dtype = torch.float16 if f16 else torch.bfloat16
    xs, w, bias, residual, _ = make(shards, rows, k, n, transpose, dtype)
    bias, residual = bias if has_bias else None, residual if has_residual else None
    plan = agmm.LinearPlan(k, n, activation=kind, rhs_transpose=transpose, f16=f16)
    ws = plan.new_workspace()
    tokens = shards * rows
    want = linear(torch.cat(xs), w, bias, residual, kind, transpose, dtype)
    buf = {name: torch.full((tokens + 3, n), 7.0, dtype=dtype, device="cuda") for name in ("out", "pre", "plain")}
    plan.run(xs, w, buf["out"][:tokens], ws, bias=bias, residual=residual, pre=buf["pre"][:tokens])
    if has_residual:
        buf["plain"][:tokens] = residual
        residual = buf["plain"][:tokens]  # in place
    plan.run(xs, w, buf["plain"][:tokens], ws, bias=bias, residual=residual)
    plan.query_status(ws)
    check(buf["out"][:tokens], *want["out"], "out")
    check(buf["pre"][:tokens], *want["pre"], "pre")
    assert torch.equal(buf["plain"][:tokens], buf["out"][:tokens])
    for name in buf:
        assert bool((buf[name][tokens:] == 7.0).all()), name


BACKWARD = [
    (1, 1, 64, 128, True, False, None, False),
    (1, 1, 1024, 4096, False, False, "gelu", False),
    (1, 7, 200, 136, True, True, "gelu_tanh", True),
    (1, 128, 264, 384, False, False, "relu", False),
    (4, 40, 136, 264, True, False, "silu", True),
    (8, 3, 72, 72, False, True, None, False),
    (1, 1003, 328, 520, False, True, "gelu", False),
    (3, 200, 512, 256, True, False, None, True),
    (1, 4096, 256, 512, True, False, "silu", False),
    (1, 640, 1280, 1536, False, False, "relu", False),
]


@pytest.mark.parametrize("case", BACKWARD, ids=ids(BACKWARD))
def test_backward(agmm, case):
    shards, rows, k, n, transpose, f16, kind, f32 = case
    dtype = torch.float16 if f16 else torch.bfloat16
    grad_dtype = torch.float32 if f32 else dtype
    xs, w, _, d, z = make(shards, rows, k, n, transpose, dtype, 1)
    z = z * 2 if kind else None
    want = linear_grad(d, torch.cat(xs), w, z, kind, transpose, dtype, grad_dtype)
    plan = agmm.LinearPlan(k, n, activation=kind, rhs_transpose=transpose, f16=f16)
    ws = plan.new_workspace()
    new = lambda *s, t=dtype: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    got = dict(dx=new(shards * rows, k), dw=new(*w.shape, t=grad_dtype), d_bias=new(n, t=grad_dtype))
    d_pre = new(*d.shape) if kind else None
    plan.backward(d, xs, w, ws, pre=z, d_pre=d_pre, **got)
    plan.query_status(ws)
    if kind:
        got["d_pre"] = d_pre
    for name, x in got.items():
        check(x, *want[name], name)
    # one at a time, and over the saved sum.  A product alone may be cut along its sum, where both
    # in one launch are not: another order of the same float32 sums, each within the bound
    for name in ("dx", "dw", "d_bias"):
        alone = torch.full_like(got[name], float("nan"))
        over = z.clone() if kind else None
        plan.backward(d, xs, w, ws, pre=over, d_pre=over, **{name: alone})
        check(alone, *want[name], name)


@pytest.mark.parametrize("kind", [None, "gelu"])
@pytest.mark.parametrize("rows, n", [(1, 8), (63, 72), (65, 1000), (257, 264), (384, 520), (385, 520)])
def test_sums_of_few_rows(agmm, rows, n, kind):
    """The bias' gradient beside the activation's, or in a launch of its own."""
    (x,), w, _, d, z = make(1, rows, 64, n, False, torch.bfloat16, 8)
    z = z * 2 if kind else None
    want = linear_grad(d, x, w, z, kind, False, torch.bfloat16, torch.float32)
    plan = agmm.LinearPlan(64, n, activation=kind)
    d_pre = torch.full((rows + 1, n), 7.0, dtype=torch.bfloat16, device="cuda")
    d_bias = torch.full((n + 8,), 7.0, device="cuda")
    plan.backward(d, x, w, plan.new_workspace(), pre=z, d_pre=d_pre[:rows] if kind else None, d_bias=d_bias[:n])
    check(d_bias[:n], *want["d_bias"], "d_bias")
    assert bool((d_bias[n:] == 7).all()) and bool((d_pre[rows:] == 7).all())
    if kind:
        check(d_pre[:rows], *want["d_pre"], "d_pre")


def test_strides(agmm):
    k, n, t = 136, 200, 150
    g = torch.Generator(device="cuda").manual_seed(4)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, r, w = new(t, k + 24)[:, 8:8 + k], new(t, n + 8)[:, :n], new(k, n + 16)[:, 16:] * 0.1
    wide = torch.full((t, 3 * n), 7.0, dtype=torch.bfloat16, device="cuda")
    plan = agmm.LinearPlan(k, n)
    plan.run(x, w, wide[:, n:2 * n], plan.new_workspace(), residual=r)
    check(wide[:, n:2 * n], *linear(x, w, None, r, None, False, torch.bfloat16)["out"], "out")
    assert bool((wide[:, :n] == 7).all()) and bool((wide[:, 2 * n:] == 7).all())


def test_broadcast_gradient(agmm):
    """The gradient of a sum is one value for all; the functions read it where rows do not lie apart."""
    xs, w, bias, _, _ = make(1, 37, 72, 136, True, torch.bfloat16, 3)
    d = torch.ones((), dtype=torch.bfloat16, device="cuda").expand(37, 136)
    out, pre = agmm.linear_matmul(xs, w, bias=bias, activation="silu", rhs_transpose=True, return_saved=True)
    dx, dw, db = agmm.linear_matmul_backward(d, xs, w, pre=pre, activation="silu", rhs_transpose=True)
    want = linear_grad(d, xs[0], w, pre, "silu", True, torch.bfloat16, torch.bfloat16)
    for name, x in dict(dx=dx, dw=dw, d_bias=db).items():
        check(x, *want[name], name)


def test_no_tokens(agmm):
    plan = agmm.LinearPlan(64, 128, rhs_transpose=True)
    ws = plan.new_workspace()
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(128, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    plan.run(x, w, none, ws, residual=none)
    dw, db = torch.full((128, 72), 5.0, device="cuda")[:, :64], torch.full((128,), 5.0, device="cuda")
    plan.backward(none, x, w, ws, dx=x, dw=dw, d_bias=db)
    assert not bool(dw.any()) and not bool(db.any())


def test_repeats_are_equal(agmm):
    """Cut tiles are added in one order, whoever comes last."""
    for rows in (1, 40, 300):
        xs, w, bias, r, _ = make(1, rows, 8192, 256, True, torch.bfloat16, 6)
        plan = agmm.LinearPlan(8192, 256, rhs_transpose=True)
        ws = plan.new_workspace()
        first = torch.empty_like(r)
        plan.run(xs, w, first, ws, bias=bias, residual=r)
        for _ in range(20):
            again = torch.empty_like(r)
            plan.run(xs, w, again, ws, bias=bias, residual=r)
            assert torch.equal(first, again)
