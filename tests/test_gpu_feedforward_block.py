"""The operators of the feed-forward half together: the example, its gradients, and the
whole of it captured in a graph."""
import os
import runpy
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def agmm():
    import all_gather_gemm_agmm_gb300 as m
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    m.load_library()
    return m


def test_example_runs(agmm, capsys):
    runpy.run_path(os.path.join(ROOT, "examples", "feed_forward_block.py"), run_name="__main__")
    assert "one token alone" in capsys.readouterr().out


@pytest.fixture(scope="module")
def example(agmm):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import feed_forward_block

    return feed_forward_block


@pytest.mark.parametrize("tokens", [1, 5, 64, 300])
def test_gradients_of_the_block(example, tokens):
    """Each of the chain's matrices is rounded to 8 bits, relatively 2^-8 at most and 2^-8 / sqrt(3) on
    average; a gradient has at most 12 of them behind it (x, norm, its weights, gate, up, out, d_out, their
    gradients), which are independent: sqrt(12 / 3) 2^-8 = 0.8 % of its norm.  Held to 2 %."""
    pairs, _, _ = example.gradients(tokens, seed=tokens)
    for name, (a, b) in pairs.items():
        assert a.shape == b.shape
        assert float((a.double() - b).norm() / b.norm()) < 2e-2, name


def test_gradients_against_differences(example):
    """Along a direction, the kernels' gradient is the slope of the block in 64 bits."""
    pairs, x, params = example.gradients(40, seed=9)
    g = torch.Generator(device="cuda").manual_seed(3)
    d = torch.Generator(device="cuda").manual_seed(9)
    torch.randn((40, example.HIDDEN), generator=d, device="cuda")  # as the example draws it: x, then d
    d = torch.randn((40, example.HIDDEN), generator=d, device="cuda").bfloat16().double()
    leaves = [x.double()] + [p.detach().double() for p in params]
    h = 1e-4
    for i, name in enumerate(("x",) + example.NAMES):
        # along the gradient itself, so that the slope is its norm
        v = pairs[name][0].double()
        v = v / v.norm() * leaves[i].norm() + 0.1 * torch.randn(v.shape, generator=g, device="cuda", dtype=torch.float64)
        moved = [[y + s * h * v if j == i else y for j, y in enumerate(leaves)] for s in (1, -1)]
        with torch.no_grad():
            slope = float(((example.block64(moved[0][0], moved[0][1:]) - example.block64(moved[1][0], moved[1][1:])) * d).sum()) / (2 * h)
        got = float((pairs[name][0].double() * v).sum())
        assert abs(got - slope) <= 2e-2 * float(pairs[name][0].double().norm() * v.norm()), name


def test_block_in_a_graph(agmm):
    """Forward and backward of all three captured on a side stream while eager calls of the same
    buffers live, then replayed with other inputs: as eager calls give them."""
    t, k, n = 200, 264, 520
    g = torch.Generator(device="cuda").manual_seed(5)
    new = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    x, d, w, b = new(t, k), new(t, k), new(k), new(k)
    wg, wu, wd = new(n, k, std=k ** -0.5), new(n, k, std=k ** -0.5), new(k, n, std=n ** -0.5)
    norm, gated, down = agmm.LayerNormPlan(k), agmm.GatedPlan(k, n, rhs_transpose=True), agmm.LinearPlan(n, k, rhs_transpose=True)

    class Buffers:
        def __init__(self):
            self.ws, self.norm_ws = gated.new_workspace(), norm.new_workspace()
            e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
            self.h, self.dh, self.dx, self.y = e(t, k), e(t, k), e(t, k), e(t, k)
            self.mean, self.rstd = (torch.empty(t, device="cuda") for _ in range(2))
            self.a, self.gate, self.up, self.da, self.dg, self.du = (e(t, n) for _ in range(6))
            self.dwg, self.dwu, self.dwd = e(n, k), e(n, k), e(k, n)
            self.dw, self.db = e(k), e(k)

        def run(self, stream=None):
            norm.run(x, self.h, weight=w, bias=b, mean=self.mean, rstd=self.rstd, stream=stream)
            gated.run(self.h, wg, wu, self.a, self.ws, gate=self.gate, up=self.up, stream=stream)
            down.run(self.a, wd, self.y, self.ws, residual=x, stream=stream)
            down.backward(d, self.a, wd, self.ws, dx=self.da, dw=self.dwd, stream=stream)
            gated.backward(self.da, self.h, wg, wu, self.gate, self.up, self.dg, self.du, self.ws, dx=self.dh, dw_gate=self.dwg,
                           dw_up=self.dwu, stream=stream)
            norm.backward(self.dh, x, self.mean, self.rstd, self.dx, self.norm_ws, weight=w, add=d, d_weight=self.dw, d_bias=self.db,
                          stream=stream)

        def results(self):
            return [self.y, self.dx, self.dw, self.db, self.dwg, self.dwu, self.dwd]

    eager, captured = Buffers(), Buffers()
    eager.run()
    captured.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.run()
    for seed in range(3):
        g.manual_seed(100 + seed)
        x.copy_(new(t, k))
        d.copy_(new(t, k))
        for r in captured.results():
            r.fill_(float("nan"))
        graph.replay()
        eager.run()
        torch.cuda.synchronize()
        for p, q in zip(eager.results(), captured.results()):
            assert torch.equal(p, q)
    gated.query_status(captured.ws)
