"""Feed-forward products that save what the backward pass reads in float32: the same results, what is
saved is what the 16-bit plan rounds, and gradients without that rounding."""
import pytest
import torch

from feedforward_ref import check, gated, gated_grad, linear, linear_grad

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def agmm():
    import all_gather_gemm_agmm_gb300 as m
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    m.load_library()
    return m


VARIANTS = [dict(AGMM_PATH="1", AGMM_SPLITK="1"), dict(AGMM_PATH="1", AGMM_SPLITK="5")]
VARIANTS += [dict(AGMM_PATH="0", AGMM_BN=bn, AGMM_STREAMK=cut) for bn in ("128", "256") for cut in ("0", "1")]
VARIANTS += [dict(AGMM_PATH="0", AGMM_BN="128", AGMM_SPLITK="3")]


def name(env):
    return "-".join(k[5:].lower() + v for k, v in env.items())


def padded(rows, cols, dtype, value=7.0):
    """(a matrix inside a larger one, the larger one)"""
    base = torch.full((rows + 2, cols + 24), value, dtype=dtype, device="cuda")
    return base[:rows, 8:8 + cols], base


def untouched(base, x):
    rest = torch.ones(base.shape, dtype=torch.bool, device="cuda")
    rest[:x.shape[0], 8:8 + x.shape[1]] = False
    return bool((base[rest] == 7).all())


@pytest.mark.parametrize("env", VARIANTS, ids=name)
@pytest.mark.parametrize("size", [(1, 1, 1000, 264), (3, 13, 584, 136), (2, 200, 1032, 648)], ids=str)
@pytest.mark.parametrize("f16", [False, True])
def test_forward(agmm, monkeypatch, env, size, f16):
    shards, rows, k, n = size
    if env["AGMM_PATH"] == "1" and shards * (-(-rows // 8) * 8) > 64:
        pytest.skip("more tokens than a swapped tile has")
    for e, v in env.items():
        monkeypatch.setenv(e, v)
    dtype, t = (torch.float16 if f16 else torch.bfloat16), shards * rows
    g = torch.Generator(device="cuda").manual_seed(21)
    new = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
    xs, wg, wu, b, r = [new(rows, k) for _ in range(shards)], new(n, k, std=k ** -0.5), new(n, k, std=k ** -0.5), new(n), new(t, n)
    got = []
    for f32 in (False, True):
        saved = F32 if f32 else dtype
        plan = agmm.GatedPlan(k, n, rhs_transpose=True, f16=f16, f32_saved=f32)
        ws = plan.new_workspace()
        (out, o), (gate, p), (up, q) = padded(t, n, dtype), padded(t, n, saved), padded(t, n, saved)
        plan.run(xs, wg, wu, out, ws, gate=gate, up=up)
        plan.query_status(ws)
        assert untouched(o, out) and untouched(p, gate) and untouched(q, up)
        plan = agmm.LinearPlan(k, n, activation="gelu", rhs_transpose=True, f16=f16, f32_saved=f32)
        (y, o), (pre, p), (bare, q) = padded(t, n, dtype), padded(t, n, saved), padded(t, n, saved)
        plan.run(xs, wg, y, ws, bias=b, residual=r, pre=pre)
        assert untouched(o, y) and untouched(p, pre)
        over = r.clone()  # the result in the residual's place
        plan.run(xs, wg, over, ws, residual=over, pre=bare)
        assert untouched(q, bare)
        plan.query_status(ws)
        got.append((out, gate, up, y, pre, over, bare))
    for a, c in zip(*got):
        assert torch.equal(a, c.to(dtype))
    x = torch.cat(xs)
    want = gated(x, wg, wu, "silu", True, F32)
    check(got[1][1], *want["gate"], "gate")
    check(got[1][2], *want["up"], "up")
    check(got[1][4], *linear(x, wg, b, r, "gelu", True, F32)["pre"], "pre")
    check(got[1][6], *linear(x, wg, None, r, "gelu", True, F32)["pre"], "pre without a bias")


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("rows, k, n", [(1, 64, 8), (37, 264, 1000), (384, 72, 520), (385, 72, 520), (1003, 136, 264)])
def test_backward(agmm, rows, k, n, kind):
    """Saved values that 16 bits do not hold; sums of few rows in one launch, and in parts."""
    f16 = rows % 2 == 1
    dtype = torch.float16 if f16 else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(22)
    new = lambda *s, std=1.0, t=dtype: (torch.randn(s, generator=g, device="cuda") * std).to(t)  # noqa: E731
    x, wg, wu, d = new(rows, k), new(k, n, std=k ** -0.5), new(k, n, std=k ** -0.5), new(rows, n)
    gate, up = new(rows, n + 8, std=2.0, t=F32)[:, :n], new(rows, n + 8, t=F32)[:, :n]
    plan = agmm.GatedPlan(k, n, activation=kind, f16=f16, f32_saved=True)
    ws = plan.new_workspace()
    got = dict(d_gate=torch.empty_like(d), d_up=torch.empty_like(d), dx=torch.empty_like(x), dw_gate=torch.empty_like(wg), dw_up=torch.empty_like(wg))
    plan.backward(d, x, wg, wu, gate, up, got["d_gate"], got["d_up"], ws, dx=got["dx"], dw_gate=got["dw_gate"], dw_up=got["dw_up"])
    want = gated_grad(d, x, wg, wu, gate, up, kind, False, dtype, dtype)
    for key, y in got.items():
        check(y, *want[key], key)
    plan = agmm.LinearPlan(k, n, activation=kind, f16=f16, f32_saved=True)
    got = dict(dx=torch.empty_like(x), dw=torch.empty(k, n, device="cuda"), d_bias=torch.empty(n, device="cuda"))
    over = d.clone()  # d_pre in d_out's place
    plan.backward(over, x, wg, ws, pre=gate, d_pre=over, **got)
    plan.query_status(ws)
    want = linear_grad(d, x, wg, gate, kind, False, dtype, F32)
    for key, y in dict(got, d_pre=over).items():
        check(y, *want[key], key)


def test_gradients_come_closer(agmm):
    """With float32 gradients of the weights a training step rounds gate and up (independently of one another
    and of d_gate), and d_gate and d_up; each adds U / sqrt(3) of its size on average, so the error falls to
    about sqrt(1 / 2) to sqrt(1 / 3) of itself.  Held to 0.8."""
    g = torch.Generator(device="cuda").manual_seed(23)
    new = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    t, k, n = 512, 512, 1024
    x, wg, wu, d = new(t, k), new(n, k, std=2 * k ** -0.5), new(n, k, std=k ** -0.5), new(t, n)
    x64, w64, v64 = (y.double().requires_grad_() for y in (x, wg, wu))
    (torch.nn.functional.silu(x64 @ w64.t()) * (x64 @ v64.t())).backward(d.double())
    off = {}
    for f32 in (False, True):
        _, gate, up = agmm.gated_matmul(x, wg, wu, rhs_transpose=True, return_saved=True, f32_saved=f32)
        assert gate.dtype == up.dtype == (F32 if f32 else torch.bfloat16)
        _, dwg, dwu = agmm.gated_matmul_backward(d, x, wg, wu, gate, up, rhs_transpose=True, f32_grads=True)
        off[f32] = [float((y.double() - z.grad).norm() / z.grad.norm()) for y, z in ((dwg, w64), (dwu, v64))]
    for less, more in zip(off[True], off[False]):
        assert less < 0.8 * more, off


def test_products_past_fp16_stay_finite(agmm):
    """Beyond 65504 a float32 product is saved as it is, and its gradient is finite."""
    k, n = 8, 8
    x = torch.zeros(2, k, dtype=torch.float16, device="cuda")
    x[:, 0], x[:, 1] = torch.tensor([-60000.0, 60000.0], device="cuda"), 1
    wg, wu = (torch.zeros(k, n, dtype=torch.float16, device="cuda") for _ in range(2))
    wg[0], wu[1] = 2, 0.5
    out, gate, up = agmm.gated_matmul(x, wg, wu, return_saved=True, f32_saved=True)
    assert gate[:, 0].tolist() == [-120000, 120000] and bool((up == 0.5).all()) and out[:, 0].tolist() == [0, 60000]
    d = torch.full_like(out, 0.5)
    plan = agmm.GatedPlan(k, n, f16=True, f32_saved=True)
    dg, du = torch.empty_like(d), torch.empty_like(d)
    plan.backward(d, x, wg, wu, gate, up, dg, du, plan.new_workspace())
    assert dg[:, 0].tolist() == [0, 0.25] and du[:, 0].tolist() == [0, 60000]


def test_functions_and_graphs(agmm):
    """linear_matmul and its gradient by way of the functions, captured and replayed."""
    g = torch.Generator(device="cuda").manual_seed(24)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, b, d = new(70, 136), new(264, 136), new(264), new(70, 264)

    def step():
        out, pre = agmm.linear_matmul(x, w, b, activation="gelu", rhs_transpose=True, return_saved=True, f32_saved=True)
        return (out, pre) + agmm.linear_matmul_backward(d, x, w, pre=pre, activation="gelu", rhs_transpose=True)

    want = step()
    assert want[1].dtype is F32
    check(want[3], *linear_grad(d, x, w, want[1], "gelu", True, torch.bfloat16, torch.bfloat16)["dw"], "dw")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for y in got:
            y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_rows_far_apart(agmm):
    """Rows of 4 MiB: the last one starts behind 2^33 bytes."""
    stride, rows, k, n = 1 << 20, 2051, 72, 136
    g = torch.Generator(device="cuda").manual_seed(25)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, d = new(rows, k), new(k, n), new(rows, n)
    plan = agmm.LinearPlan(k, n, activation="silu", f32_saved=True)
    ws = plan.new_workspace()
    apart = torch.empty(rows * stride, device="cuda").view(rows, stride)[:, :n]
    results = []
    for pre in (torch.empty(rows, n, device="cuda"), apart):
        out, d_pre, dx = torch.empty_like(d), torch.empty_like(d), torch.empty_like(x)
        plan.run(x, w, out, ws, pre=pre)
        plan.backward(d, x, w, ws, pre=pre, d_pre=d_pre, dx=dx)
        results.append((out, pre, d_pre, dx))
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_refusals(agmm):
    k, n, t = 64, 128, 10
    x, w, d, wide = (torch.ones(*s, dtype=torch.bfloat16, device="cuda") for s in ((t, k), (k, n), (t, n), (t, n)))
    f32 = torch.ones(t, n, device="cuda")
    for saved, right, wrong in ((False, wide, f32), (True, f32, wide)):
        plan = agmm.GatedPlan(k, n, f32_saved=saved)
        ws = plan.new_workspace()
        for gate, up in ((wrong, wrong), (right, wrong), (wrong, right)):
            with pytest.raises(ValueError, match="gate|up"):
                plan.run(x, w, w, d, ws, gate=gate, up=up)
            with pytest.raises(ValueError, match="gate|up"):
                plan.backward(d, x, w, w, gate, up, wide, wide.clone(), ws)
        plan = agmm.LinearPlan(k, n, activation="relu", f32_saved=saved)
        with pytest.raises(ValueError, match="pre"):
            plan.run(x, w, d, ws, pre=wrong)
        with pytest.raises(ValueError, match="pre"):
            plan.backward(d, x, w, ws, pre=wrong, d_pre=wide)
        with pytest.raises(ValueError, match="d_pre"):
            plan.backward(d, x, w, ws, pre=right, d_pre=f32)
    over = torch.ones(t, 2 * n, dtype=torch.bfloat16, device="cuda")[:, :n]  # float32 rows of n, seen as 16-bit ones
    f32 = over.as_strided((t, 2 * n), (2 * n, 1)).view(F32)
    with pytest.raises(agmm.AgmmError, match="float32"):
        agmm.LinearPlan(k, n, activation="relu", f32_saved=True).backward(d, x, w, ws, pre=f32, d_pre=over)
    gated = agmm.GatedPlan(k, n, f32_saved=True)
    for grads in ((over, wide), (wide, over)):
        with pytest.raises(agmm.AgmmError, match="float32"):
            plain = [torch.empty_like(over.as_strided((t, 2 * n), (2 * n, 1)))[:, :n] if y is wide else y for y in grads]
            gated.backward(d, x, w, w, f32, f32.clone(), *plain, ws)
    plan = agmm.LinearPlan(k, n)
    with pytest.raises(agmm.AgmmError, match="none"):
        plan.backward(d, x, w, ws, pre=wide)
