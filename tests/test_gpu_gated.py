"""The gated product and its backward pass against the 64-bit formulas: tokens from
none to many, shards, both layouts of the weights, both types, every activation,
odd sizes and strides."""
import pytest
import torch

from feedforward_ref import check, gated, gated_grad

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
    shape = (n, k) if transpose else (k, n)
    xs = [new(rows, k) for _ in range(shards)]
    return xs, new(*shape, std=k ** -0.5), new(*shape, std=k ** -0.5), new(shards * rows, n)


# shards, rows, k, n, [n, k], fp16, activation
FORWARD = [
    (1, 1, 64, 128, True, False, "silu"),
    (1, 1, 4096, 1024, True, False, "silu"),      # cut along k, one token
    (1, 1, 8, 8, False, True, "gelu"),            # the smallest there is
    (1, 5, 200, 136, False, False, "gelu_tanh"),
    (1, 17, 1288, 2056, True, True, "relu"),
    (1, 128, 512, 384, False, True, "silu"),      # the most tokens of swapped tiles
    (1, 129, 512, 384, True, False, "silu"),      # the fewest of row tiles
    (3, 1, 256, 128, True, False, "silu"),
    (8, 16, 1024, 264, False, False, "gelu"),
    (8, 17, 320, 200, True, False, "gelu_tanh"),  # 8 padded shards are past one swapped tile
    (5, 100, 256, 384, False, True, "silu"),      # boxes that end inside row tiles
    (2, 300, 72, 520, True, False, "silu"),
    (1, 1000, 136, 1000, False, False, "gelu"),
    (1, 257, 2048, 256, True, False, "silu"),     # few row tiles, cut along k
    (1, 2500, 512, 2304, True, True, "silu"),     # more tiles than clusters, a ragged last wave
]


def ids(cases):
    return ["x".join(str(int(v) if isinstance(v, bool) else v) for v in c) for c in cases]


@pytest.mark.parametrize("case", FORWARD, ids=ids(FORWARD))
def test_forward(agmm, case):
    shards, rows, k, n, transpose, f16, kind = case
    dtype = torch.float16 if f16 else torch.bfloat16
    xs, wg, wu, _ = make(shards, rows, k, n, transpose, dtype)
    plan = agmm.GatedPlan(k, n, activation=kind, rhs_transpose=transpose, f16=f16)
    ws = plan.new_workspace()
    tokens = shards * rows
    want = gated(torch.cat(xs), wg, wu, kind, transpose, dtype)
    guard = 3  # rows behind the last token stay as they were
    buf = {name: torch.full((tokens + guard, n), 7.0, dtype=dtype, device="cuda") for name in ("out", "gate", "up", "plain")}
    plan.run(xs, wg, wu, buf["out"][:tokens], ws, gate=buf["gate"][:tokens], up=buf["up"][:tokens])
    plan.run(xs, wg, wu, buf["plain"][:tokens], ws)  # the same workspace again, nothing saved
    plan.query_status(ws)
    for name in ("out", "gate", "up"):
        check(buf[name][:tokens], *want[name], name)
    assert torch.equal(buf["plain"][:tokens], buf["out"][:tokens])
    for name in buf:
        assert bool((buf[name][tokens:] == 7.0).all()), name


BACKWARD = [
    (1, 1, 64, 128, True, False, "silu", False),
    (1, 1, 1024, 4096, False, False, "gelu", False),  # one token: the sum over n is cut
    (1, 7, 200, 136, True, True, "gelu_tanh", True),
    (1, 128, 264, 384, False, False, "relu", False),
    (4, 40, 136, 264, True, False, "silu", True),     # shards that end inside a k block
    (8, 3, 72, 72, False, True, "silu", False),
    (1, 1003, 328, 520, False, True, "gelu", False),
    (3, 200, 512, 256, True, False, "gelu_tanh", False),
    (1, 4096, 256, 512, True, False, "silu", True),   # few tiles of weights, cut along the tokens
    (1, 640, 1280, 1536, False, False, "silu", False),
]


@pytest.mark.parametrize("case", BACKWARD, ids=ids(BACKWARD))
def test_backward(agmm, case):
    shards, rows, k, n, transpose, f16, kind, f32 = case
    dtype, grad_dtype = (torch.float16 if f16 else torch.bfloat16), None
    grad_dtype = torch.float32 if f32 else dtype
    xs, wg, wu, d = make(shards, rows, k, n, transpose, dtype, 1)
    g, u = (torch.randn(shards * rows, n, device="cuda").mul_(2).to(dtype) for _ in range(2))
    want = gated_grad(d, torch.cat(xs), wg, wu, g, u, kind, transpose, dtype, grad_dtype)
    plan = agmm.GatedPlan(k, n, activation=kind, rhs_transpose=transpose, f16=f16)
    ws = plan.new_workspace()
    new = lambda *s, t=dtype: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    got = dict(d_gate=new(*d.shape), d_up=new(*d.shape), dx=new(shards * rows, k), dw_gate=new(*wg.shape, t=grad_dtype),
               dw_up=new(*wg.shape, t=grad_dtype))
    plan.backward(d, xs, wg, wu, g, u, got["d_gate"], got["d_up"], ws, dx=got["dx"], dw_gate=got["dw_gate"], dw_up=got["dw_up"])
    plan.query_status(ws)
    for name, x in got.items():
        check(x, *want[name], name)


def test_backward_over_the_saved_products(agmm):
    """d_gate and d_up may lie over gate and up; gradients that are not asked for are not computed."""
    xs, wg, wu, d = make(1, 70, 128, 264, True, torch.bfloat16, 2)
    plan = agmm.GatedPlan(128, 264, rhs_transpose=True)
    ws = plan.new_workspace()
    out, g, u = (torch.empty_like(d) for _ in range(3))
    plan.run(xs, wg, wu, out, ws, gate=g, up=u)
    dg, du, dx, dx2 = torch.empty_like(d), torch.empty_like(d), torch.empty_like(xs[0]), torch.empty_like(xs[0])
    dwg, dwu, dwg2, dwu2 = (torch.empty_like(wg) for _ in range(4))
    plan.backward(d, xs, wg, wu, g, u, dg, du, ws, dx=dx, dw_gate=dwg, dw_up=dwu)
    g2, u2 = g.clone(), u.clone()
    want = gated_grad(d, xs[0], wg, wu, g, u, "silu", True, torch.bfloat16, torch.bfloat16)
    plan.backward(d, xs, wg, wu, g, u, g, u, ws, dx=dx2)
    assert torch.equal(g, dg) and torch.equal(u, du)
    check(dx2, *want["dx"], "dx")  # alone it may be cut along its sum: another order
    plan.backward(d, xs, wg, wu, g2, u2, g2, u2, ws, dw_gate=dwg2, dw_up=dwu2)
    for name, x, y in (("dw_gate", dwg, dwg2), ("dw_up", dwu, dwu2)):
        check(x, *want[name], name)
        check(y, *want[name], name)


def test_strides_and_halves(agmm):
    """Weights that are halves of one tensor, rows with room between them."""
    k, n, t = 136, 200, 150
    g = torch.Generator(device="cuda").manual_seed(4)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x = new(t, k + 24)[:, 8:8 + k]
    both = new(k, 2 * n) * 0.1
    wg, wu = both[:, :n], both[:, n:]
    wide = torch.full((t, 3 * n + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    plan = agmm.GatedPlan(k, n)
    ws = plan.new_workspace()
    plan.run(x, wg, wu, wide[:, n:2 * n], ws)
    check(wide[:, n:2 * n], *gated(x, wg, wu, "silu", False, torch.bfloat16)["out"], "out")
    assert bool((wide[:, :n] == 7).all()) and bool((wide[:, 2 * n:] == 7).all())
    packed = new(2 * n, k) * 0.1
    out = agmm.gated_matmul(x, packed[:n], packed[n:], rhs_transpose=True)
    check(out, *gated(x, packed[:n], packed[n:], "silu", True, torch.bfloat16)["out"], "out")


def test_no_tokens(agmm):
    plan = agmm.GatedPlan(64, 128)
    ws = plan.new_workspace()
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, 128, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    plan.run(x, w, w, none, ws)
    dwg, dwu = torch.full_like(w, 5.0), torch.full((64, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    plan.backward(none, x, w, w, none, none, none, none, ws, dx=x, dw_gate=dwg, dw_up=torch.full_like(w, 5.0))
    assert not bool(dwg.any())
    both = torch.full((64, 256), 5.0, device="cuda")
    plan.backward(none, [x, x], w, w, none, none, none, none, ws, dw_gate=both[:, :128], dw_up=both[:, 128:])
    assert not bool(both.any())
    del dwu


@pytest.mark.parametrize("rows", [3, 200])
def test_non_finite_rows_stay_alone(agmm, rows):
    """An infinity or NaN in one token reaches that token's results only."""
    xs, wg, wu, d = make(2, rows, 264, 136, True, torch.bfloat16, 5)
    plan = agmm.GatedPlan(264, 136, rhs_transpose=True)
    ws = plan.new_workspace()
    out, bad = (torch.empty_like(d) for _ in range(2))
    plan.run(xs, wg, wu, out, ws)
    xs[1][0, 3], xs[1][1, 5] = float("nan"), float("inf")
    plan.run(xs, wg, wu, bad, ws)
    keep = torch.ones(2 * rows, dtype=torch.bool, device="cuda")
    keep[rows:rows + 2] = False
    assert torch.equal(out[keep], bad[keep])
    assert not bool(torch.isfinite(bad[~keep]).any())


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
def test_far_preactivations(agmm, kind):
    """Products far from zero, where an activation is 0 or its argument, and its slope 0 or 1."""
    k, n = 8, 8
    z = torch.tensor([-3e38, -1e30, -300.0, -90.0, -30.0, 30.0, 90.0, 300.0, 1e30, 3e38, 0.0, -0.0], device="cuda").bfloat16()
    x = torch.zeros(len(z), k, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = z, 1
    wg, wu = (torch.zeros(k, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wg[0], wu[1] = 1, 1
    out, g, u = agmm.gated_matmul(x, wg, wu, activation=kind, return_saved=True)
    assert torch.equal(g[:, 0].float(), z.float() + 0)
    want = torch.where(z.double() > 0, z.double(), 0.0)
    assert bool(((out[:, 0].double() - want).abs() <= 1e-9 + 2 ** -8 * want.abs()).all()), out[:, 0]
    d = torch.ones_like(out)
    plan = agmm.GatedPlan(k, n, activation=kind)
    dg, du = torch.empty_like(d), torch.empty_like(d)
    plan.backward(d, x, wg, wu, g, u, dg, du, plan.new_workspace())
    slope = torch.where(z.double() > 0, 1.0, 0.0)
    slope[-2:] = 0.0 if kind == "relu" else 0.5
    assert bool(((dg[:, 0].double() - slope).abs() <= 1e-9 + 2 ** -8 * slope).all()), dg[:, 0]
    assert torch.equal(du[:, 0], out[:, 0])


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
def test_saved_infinities(agmm, kind):
    """An fp16 product past 65504 is saved as infinite.  Below, the activation and its slope are 0,
    and so are both gradients; above, the slope is 1 and the activation's own size infinite."""
    k, n = 8, 8
    x = torch.zeros(4, k, dtype=torch.float16, device="cuda")
    x[:, 0], x[:, 1] = torch.tensor([-60000.0, 60000.0, -40000.0, 1.0], device="cuda"), 1
    wg, wu = (torch.zeros(k, n, dtype=torch.float16, device="cuda") for _ in range(2))
    wg[0], wu[1] = 2, 0.5
    out, g, u = agmm.gated_matmul(x, wg, wu, activation=kind, return_saved=True)
    assert g[:3, 0].tolist() == [float("-inf"), float("inf"), float("-inf")]
    assert out[:3, 0].tolist() == [0, 60000, 0]  # of the float32 products, half of 120000 among them
    plan = agmm.GatedPlan(k, n, activation=kind, f16=True)
    d = torch.ones_like(out)
    dg, du = torch.empty_like(d), torch.empty_like(d)
    plan.backward(d, x, wg, wu, g, u, dg, du, plan.new_workspace())
    assert dg[:3, 0].tolist() == [0, 0.5, 0]
    assert du[:3, 0].tolist() == [0, float("inf"), 0]
    assert bool(dg[3].isfinite().all() and du[3].isfinite().all())
    linear = agmm.LinearPlan(k, n, activation=kind, f16=True)
    d_pre, dx = torch.empty_like(d), torch.empty_like(x)
    linear.backward(d, x, wg, linear.new_workspace(), pre=g, d_pre=d_pre, dx=dx)
    assert d_pre[:3, 0].tolist() == [0, 1, 0]
    assert bool(dx.isfinite().all())
