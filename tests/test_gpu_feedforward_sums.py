"""Sums over millions of tokens, value by value: of whole numbers small enough that float32 holds every
partial sum exactly, so a k block, a row or a part that is missing or counted twice is seen.

2^22 + 3 tokens: 65537 k blocks of the weights' gradients, the last of 3 rows.  Terms are at most 2, so no
sum of some of them passes 2^23 + 6 < 2^24."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TOKENS = (1 << 22) + 3


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


def whole(g, most, *s):
    return torch.randint(-most, most + 1, s, generator=g, device="cuda").bfloat16()


def same(got, want):
    """want in 64 bits; got rounded once from it."""
    assert float(want.abs().max()) > 0 and float(want.abs().max()) < 2 ** 24
    assert torch.equal(got, want.float().to(got.dtype))


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("merge", ["0", "1"])
def test_linear(agmm, monkeypatch, transpose, merge, f32):
    """Both gradients in one launch, or the weights' cut along the tokens; a quarter of the products' slopes is 0."""
    monkeypatch.setenv("AGMM_MERGE", merge)
    g = torch.Generator(device="cuda").manual_seed(11)
    k, n = 8, 16
    x, d, pre = whole(g, 1, TOKENS, k), whole(g, 2, TOKENS, n), whole(g, 3, TOKENS, n)
    w = whole(g, 1, *((n, k) if transpose else (k, n)))
    plan = agmm.LinearPlan(k, n, activation="relu", rhs_transpose=transpose)
    ws = plan.new_workspace()
    dtype = torch.float32 if f32 else torch.bfloat16
    d_pre, dx = torch.empty_like(d), torch.empty_like(x)
    dw, db = torch.full(w.shape, float("nan"), dtype=dtype, device="cuda"), torch.full((n,), float("nan"), dtype=dtype, device="cuda")
    plan.backward(d, x, w, ws, pre=pre, d_pre=d_pre, dx=dx, dw=dw, d_bias=db)
    plan.query_status(ws)
    z = torch.where(pre > 0, d.double(), 0.0)
    want = x.double().t() @ z
    same(dw, want.t() if transpose else want)
    same(db, z.sum(0))
    same(d_pre, z)
    same(dx, z @ (w if transpose else w.t()).double())


def test_gated(agmm):
    """Four shards: the tokens of each are a segment of the sum, whose last k block has one row."""
    g = torch.Generator(device="cuda").manual_seed(12)
    rows, k, n = (1 << 20) + 1, 8, 16
    xs = [whole(g, 1, rows, k) for _ in range(4)]
    d, gate, up = whole(g, 1, 4 * rows, n), whole(g, 1, 4 * rows, n), whole(g, 2, 4 * rows, n)
    wg, wu = whole(g, 1, k, n), whole(g, 1, k, n)
    plan = agmm.GatedPlan(k, n, activation="relu")
    ws = plan.new_workspace()
    d_gate, d_up = torch.empty_like(d), torch.empty_like(d)
    dwg, dwu = (torch.full((k, n), float("nan"), device="cuda") for _ in range(2))
    plan.backward(d, xs, wg, wu, gate, up, d_gate, d_up, ws, dw_gate=dwg, dw_up=dwu)
    plan.query_status(ws)
    x = torch.cat(xs).double().t()
    same(dwg, x @ torch.where(gate > 0, d.double() * up.double(), 0.0))
    same(dwu, x @ torch.where(gate > 0, d.double() * gate.double(), 0.0))


@pytest.mark.parametrize("rows, columns", [(TOKENS, 16), ((1 << 17) + 5, 1032), ((1 << 15) + 7, 8200)])
def test_layer_norm(agmm, rows, columns):
    """Rows whose statistics are 0 and 1, as the backward pass is given them."""
    g = torch.Generator(device="cuda").manual_seed(13)
    x, d = whole(g, 1, rows, columns), whole(g, 2, rows, columns)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    plan = agmm.LayerNormPlan(columns)
    dw, db = (torch.full((columns,), float("nan"), device="cuda") for _ in range(2))
    plan.backward(d, x, mean, rstd, None, plan.new_workspace(), d_weight=dw, d_bias=db)
    same(dw, sum((a.double() * b.double()).sum(0) for a, b in zip(d.chunk(64), x.chunk(64))))
    same(db, sum(a.double().sum(0) for a in d.chunk(64)))
