"""Layer norm and its backward pass against the 64-bit formulas."""
import pytest
import torch

from feedforward_ref import check, norm, norm_grad

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


# rows, columns, fp16, weight, bias, add, float32 gradients
CASES = [
    (1, 8, False, True, True, False, False),
    (1, 4096, False, True, True, True, False),
    (3, 256, True, True, False, False, True),
    (7, 264, False, False, True, True, False),
    (509, 1000, True, True, True, False, False),
    (700, 1024, False, True, True, False, True),
    (130, 1032, False, True, True, True, False),
    (33, 2056, True, False, False, True, False),
    (1500, 4104, False, True, True, False, False),
    (400, 8192, False, True, True, True, False),
    (40, 8200, True, True, True, True, True),
    (200, 16384, False, True, True, False, False),
    (5000, 128, False, True, True, True, True),
]


def ids(cases):
    return ["x".join(str(int(v)) for v in c) for c in cases]


def make(rows, columns, dtype, seed=0, mean=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g, device="cuda") * std + mean).to(dtype)  # noqa: E731
    return new(rows, columns, std=1.5, mean=mean), new(columns, std=0.2, mean=1.0), new(columns), new(rows, columns), new(rows, columns)


@pytest.mark.parametrize("case", CASES, ids=ids(CASES))
def test_forward_and_backward(agmm, case):
    rows, columns, f16, has_w, has_b, has_add, f32 = case
    dtype = torch.float16 if f16 else torch.bfloat16
    grad_dtype = torch.float32 if f32 else dtype
    x, w, b, d, add = make(rows, columns, dtype)
    w, b, add = w if has_w else None, b if has_b else None, add if has_add else None
    plan = agmm.LayerNormPlan(columns, eps=1e-5, f16=f16)
    out = torch.full((rows + 2, columns), 7.0, dtype=dtype, device="cuda")
    mean, rstd = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    plan.run(x, out[:rows], weight=w, bias=b, mean=mean, rstd=rstd)
    want = norm(x, w, b, 1e-5, dtype)
    for name, got in dict(out=out[:rows], mean=mean, rstd=rstd).items():
        check(got, *want[name], name)
    assert bool((out[rows:] == 7).all())
    inplace = x.clone()
    plan.run(inplace, inplace, weight=w, bias=b)
    assert torch.equal(inplace, out[:rows])

    ws = plan.new_workspace()
    dx = torch.full((rows + 2, columns), 7.0, dtype=dtype, device="cuda")
    dw, db = (torch.full((columns,), float("nan"), dtype=grad_dtype, device="cuda") for _ in range(2))
    plan.backward(d, x, mean, rstd, dx[:rows], ws, weight=w, add=add, d_weight=dw, d_bias=db)
    want = norm_grad(d, x, mean, rstd, w, add, dtype, grad_dtype)
    for name, got in dict(dx=dx[:rows], d_weight=dw, d_bias=db).items():
        check(got, *want[name], name)
    assert bool((dx[rows:] == 7).all())
    # what is not wanted is not needed; dx may lie over d_out, or over what is added
    over, only = d.clone(), torch.full_like(dw, float("nan"))
    plan.backward(over, x, mean, rstd, over, None, weight=w, add=add)
    assert torch.equal(over, dx[:rows])
    if has_add:
        over = add.clone()
        plan.backward(d, x, mean, rstd, over, None, weight=w, add=over)
        assert torch.equal(over, dx[:rows])
    plan.backward(d, x, mean, rstd, None, ws, weight=w, d_weight=only)
    assert torch.equal(only, dw)
    plan.backward(d, x, mean, rstd, None, ws, weight=w, d_bias=only)
    assert torch.equal(only, db)


@pytest.mark.parametrize("rows, columns", [(767, 1000), (768, 8), (769, 1000), (1023, 264), (1024, 1032), (1025, 2056), (65, 16384), (13, 72)])
def test_rows_about_the_bounds_of_few(agmm, rows, columns):
    """Sums and dx in one launch, or apart; dx in d_out's place, where one launch would read it too late."""
    x, w, _, d, add = make(rows, columns, torch.bfloat16, 9)
    plan = agmm.LayerNormPlan(columns)
    _, mean, rstd = agmm.layer_norm(x, w, None, return_stats=True)
    want = norm_grad(d, x, mean, rstd, w, add, torch.bfloat16, torch.float32)
    ws = plan.new_workspace()
    for over in (False, True):
        dw, db = (torch.full((columns,), float("nan"), device="cuda") for _ in range(2))
        d_out = torch.full((rows, columns + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        d_out[:, :columns] = d
        dx = d_out[:, :columns] if over else torch.full_like(d, float("nan"))
        plan.backward(d_out[:, :columns], x, mean, rstd, dx, ws, weight=w, add=add, d_weight=dw, d_bias=db)
        for name, got in dict(dx=dx, d_weight=dw, d_bias=db).items():
            check(got, *want[name], name)
        assert bool((d_out[:, columns:] == 7).all())


def test_values_about_a_far_mean(agmm):
    """Rows far from zero: the squares are taken about the mean."""
    x, w, b, _, _ = make(20, 2048, torch.float16, 3, mean=300.0)
    out, mean, rstd = agmm.layer_norm(x, w, b, return_stats=True)
    want = norm(x, w, b, 1e-5, torch.float16)
    for name, got in dict(out=out, mean=mean, rstd=rstd).items():
        check(got, *want[name], name)


def test_constant_rows(agmm):
    x = torch.full((5, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    out, mean, rstd = agmm.layer_norm(x, None, None, return_stats=True)
    assert not bool(out.any()) and bool((mean == 3).all())
    check(rstd, torch.full((5,), 1e-5 ** -0.5, dtype=torch.float64, device="cuda"), torch.full((5,), 1e-3, device="cuda"), "rstd")


def test_strides_and_rows_that_stay_alone(agmm):
    g = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn(60, 3 * 520, generator=g, device="cuda").bfloat16()
    x = wide[:, 520:1040]
    out = torch.full((60, 528), 7.0, dtype=torch.bfloat16, device="cuda")
    plan = agmm.LayerNormPlan(520)
    plan.run(x, out[:, :520])
    check(out[:, :520], *norm(x, None, None, 1e-5, torch.bfloat16)["out"], "out")
    assert bool((out[:, 520:] == 7).all())
    before = out[:, :520].clone()
    x[7, 3] = float("nan")
    plan.run(x, out[:, :520])
    assert bool(out[7, :520].isnan().all())
    keep = torch.arange(60, device="cuda") != 7
    assert torch.equal(out[keep, :520], before[keep])


def test_no_rows(agmm):
    plan = agmm.LayerNormPlan(64)
    x, s = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, device="cuda")
    plan.run(x, x, mean=s, rstd=s)
    dw, db = (torch.full((64,), 5.0, device="cuda") for _ in range(2))
    plan.backward(x, x, s, s, x, plan.new_workspace(), d_weight=dw, d_bias=db)
    assert not bool(dw.any()) and not bool(db.any())
