"""What the feed-forward operators refuse: by name of the argument, before anything is launched."""
import pytest
import torch

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


def new(*s, dtype=torch.bfloat16):
    return torch.ones(s, dtype=dtype, device="cuda")


def refused(call, word, kind=Exception):
    with pytest.raises(kind, match=word):
        call()


def test_products(agmm):
    k, n, t = 64, 128, 10
    for plan in (agmm.GatedPlan(k, n), agmm.LinearPlan(k, n)):
        gated = isinstance(plan, agmm.GatedPlan)
        ws = plan.new_workspace()
        x, w, out = new(t, k), new(k, n), torch.full((t, n), 7.0, dtype=torch.bfloat16, device="cuda")

        def run(x=x, w=w, out=out, ws=ws, **kw):
            plan.run(x, *([w, kw.pop("w2", w)] if gated else [w]), out, ws, **kw)

        refused(lambda: run(x=x.half()), "X")
        refused(lambda: run(x=x.cpu()), "X")
        refused(lambda: run(x=new(t, k + 8)), "X")
        refused(lambda: run(x=new(k, t).t()), "X")
        refused(lambda: run(x=[x, new(t + 1, k)]), "X")
        refused(lambda: run(x=[x] * 9), "shards")
        refused(lambda: run(x=[]), "shards")
        refused(lambda: run(x=[x, new(t, 2 * k)[:, :k]]), "row stride")
        refused(lambda: run(w=new(n, k)), "w")
        refused(lambda: run(w=w.half()), "w")
        refused(lambda: run(out=new(t + 1, n)), "out")
        refused(lambda: run(out=new(t, n, dtype=torch.float32)), "out")
        refused(lambda: run(out=new(t, n + 4)[:, :n]), "multiple of 8")
        refused(lambda: run(out=new(t, n + 8)[:, 4:n + 4]), "aligned")
        refused(lambda: run(x=new(1, k).expand(t, k)), "row stride")
        refused(lambda: run(ws=ws[:1000]), "workspace")
        refused(lambda: run(ws=torch.empty(ws.numel() + 64, dtype=torch.uint8, device="cuda")[64:]), "workspace")
        refused(lambda: run(w=new(k, n).requires_grad_()), "requires grad")
        with torch.no_grad():
            run(w=new(k, n).requires_grad_(), out=new(t, n))
        if gated:
            refused(lambda: run(gate=new(t, n)), "together")
            refused(lambda: run(gate=new(t, n), up=new(t, n + 8)[:, :n]), "row stride")
            refused(lambda: run(w2=new(k, 2 * n)[:, :n]), "row stride")
        else:
            refused(lambda: run(bias=new(n + 8)), "bias")
            refused(lambda: run(bias=new(2 * n)[::2]), "bias")
            refused(lambda: run(residual=new(t, k)), "residual")
            refused(lambda: run(pre=new(t, k)), "pre")
        torch.cuda.synchronize()
        assert bool((out == 7).all())


def test_backward_passes(agmm):
    k, n, t = 64, 128, 10
    plan = agmm.GatedPlan(k, n)
    ws = plan.new_workspace()
    x, w, d = new(t, k), new(k, n), new(t, n)

    def back(d=d, g=d, dg=None, **kw):
        dg = new(t, n) if dg is None else dg
        plan.backward(d, x, w, w, g, d, dg, dg, ws, **kw)

    refused(lambda: back(d=new(t, k)), "d_out")
    refused(lambda: back(g=new(t, n, dtype=torch.float32)), "gate")
    refused(lambda: back(dg=new(t, k)), "d_gate")
    refused(lambda: back(dx=new(t, n)), "dx")
    refused(lambda: back(dw_gate=new(k, n)), "together")
    refused(lambda: back(dw_gate=new(k, n), dw_up=new(k, n, dtype=torch.float32)), "all float32")
    refused(lambda: back(dw_gate=new(n, k), dw_up=new(n, k)), "dw_gate")
    refused(lambda: back(dw_gate=new(k, n, dtype=torch.float16), dw_up=new(k, n, dtype=torch.float16)), "dw_gate")

    plan = agmm.LinearPlan(k, n)
    refused(lambda: plan.backward(d, x, w, ws, pre=d, dx=new(t, k)), "none")
    refused(lambda: plan.backward(d, x, w, ws, dw=new(k, n), d_bias=new(n, dtype=torch.float32)), "all float32")
    refused(lambda: plan.backward(d, x, w, ws, d_bias=new(k)), "d_bias")
    plan = agmm.LinearPlan(k, n, activation="silu")
    refused(lambda: plan.backward(d, x, w, ws, dx=new(t, k)), "pre")
    refused(lambda: plan.backward(d, x, w, ws, pre=d, dx=new(t, k)), "d_pre")

    plan = agmm.LayerNormPlan(k)
    ws = plan.new_workspace()
    s = new(t, dtype=torch.float32)
    refused(lambda: plan.run(x, x, weight=new(k, dtype=torch.float32)), "weight")
    refused(lambda: plan.run(x, x, mean=new(t)), "mean")
    refused(lambda: plan.run(x, new(t, k + 4)[:, :k]), "multiple of 8")
    refused(lambda: plan.run(new(t, k + 8), x), "x")
    refused(lambda: plan.backward(x, x, s, s, None, ws, add=x, d_weight=new(k)), "add")
    refused(lambda: plan.backward(x, x, s, s[:3], x, ws), "rstd")
    refused(lambda: plan.backward(x, x, s, s, x, None, d_weight=new(k)), "workspace|NoneType")
    refused(lambda: plan.backward(x, x, s, s, x, ws, d_weight=new(k), d_bias=new(k, dtype=torch.float32)), "all float32")


def test_functions(agmm):
    x, w = new(10, 64), new(64, 128)
    refused(lambda: agmm.gated_matmul(x, new(72, 128), new(72, 128)), "contracting")
    refused(lambda: agmm.gated_matmul(x, w, w, activation=None), "activation")
    refused(lambda: agmm.gated_matmul(x.float(), w.float(), w.float()), "bfloat16 or float16")
    refused(lambda: agmm.linear_matmul([], w), "list of such shards")
    refused(lambda: agmm.layer_norm(new(4, 4, 64)), "rows, columns")
    refused(lambda: agmm.layer_norm(new(4, 60)), "columns")
    refused(lambda: agmm.linear_matmul(x, w.requires_grad_()), "requires grad")


def test_functions_take_any_rows(agmm):
    """Transposed and offset tensors are copied; the plans' own calls refuse them."""
    x, w = torch.randn(64, 20, device="cuda").bfloat16().t(), torch.randn(128, 64, device="cuda").bfloat16()
    assert torch.equal(agmm.linear_matmul(x, w.t()), agmm.linear_matmul(x.contiguous(), w, rhs_transpose=True))
    wide = torch.randn(20, 68, device="cuda").bfloat16()
    assert torch.equal(agmm.layer_norm(wide[:, 4:]), agmm.layer_norm(wide[:, 4:].contiguous()))
    a, b = torch.randn(2, 64, 128, device="cuda").bfloat16(), torch.randn(64, 136, device="cuda").bfloat16()[:, :128]
    assert torch.equal(agmm.gated_matmul([x, x], a[0], b), agmm.gated_matmul(torch.cat([x, x]), a[0], b.contiguous()))
