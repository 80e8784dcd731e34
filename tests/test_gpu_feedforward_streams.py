"""The feed-forward operators on other streams, several at once, in graphs, and with buffers
that held other bytes before."""
import pytest
import torch

pytestmark = pytest.mark.gpu


class Handle:
    """Another library's stream object."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


FORMS = {
    "stream": lambda s: s,
    "handle": lambda s: s.cuda_stream,
    "object": Handle,
}


@pytest.fixture(scope="module")
def agmm():
    import all_gather_gemm_agmm_gb300 as m
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    m.load_library()
    return m


def calls(agmm):
    g = torch.Generator(device="cuda").manual_seed(2)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, v, d, b, r = new(300, 2056), new(264, 2056) * 0.02, new(264, 2056) * 0.02, new(300, 264), new(264), new(300, 264)
    one = x[:1].clone()
    t, weight = new(700, 520), new(520)
    y, mean, rstd = agmm.layer_norm(t, weight, return_stats=True)
    out, gate, up = agmm.gated_matmul(x, w, v, rhs_transpose=True, return_saved=True)
    torch.cuda.synchronize()
    return {
        "norm": lambda **kw: agmm.layer_norm(t, weight, return_stats=True, **kw),
        "norm backward": lambda **kw: agmm.layer_norm_backward(y, t, mean, rstd, weight, **kw),
        "gated": lambda **kw: (agmm.gated_matmul(x, w, v, rhs_transpose=True, **kw),),
        "gated token": lambda **kw: (agmm.gated_matmul(one, w, v, rhs_transpose=True, **kw),),
        "gated backward": lambda **kw: agmm.gated_matmul_backward(d, x, w, v, gate, up, rhs_transpose=True, **kw),
        "linear": lambda **kw: (agmm.linear_matmul(x, w, b, r, "gelu", True, **kw),),
        "linear backward": lambda **kw: agmm.linear_matmul_backward(d, x, w, gate, "gelu", True, **kw),
    }


NAMES = ["norm", "norm backward", "gated", "gated token", "gated backward", "linear", "linear backward"]


def same(got, want):
    return len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def dirty():
    """Free blocks of the current stream that hold large numbers, for workspaces and outputs to be made in."""
    for mb in (1, 2, 4, 8, 16, 32, 40, 48, 64):
        torch.full((mb << 20,), 0x3f, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("name", NAMES)
def test_buffers_belong_to_the_given_stream(agmm, name, form):
    call = calls(agmm)[name]
    want = call()
    dirty()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    busy = torch.cuda.Event()
    busy.record()
    got = call(stream=FORMS[form](s))
    s.synchronize()
    assert not busy.query(), "the call waited for the current stream"
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_buffers_that_held_other_bytes(agmm, name):
    call = calls(agmm)[name]
    want = call()
    for _ in range(3):
        dirty()
        assert same(call(), want)


@pytest.mark.parametrize("name", NAMES)
def test_captured_calls(agmm, name):
    """A call captured with buffers of the graph's own, replayed; two graphs, one after the other."""
    call = calls(agmm)[name]
    want = call()
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(call())
    for _ in range(3):
        for graph, out in zip(graphs, outs):
            for o in out:
                o.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert same(out, want)


def test_two_streams_at_once(agmm):
    """One plan on two streams, each with a workspace of its own, many times."""
    g = torch.Generator(device="cuda").manual_seed(4)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, y, w = new(300, 4096), new(1, 4096), new(264, 4096)
    plan = agmm.LinearPlan(4096, 264, activation="silu", rhs_transpose=True)
    ws = [plan.new_workspace() for _ in range(2)]
    want = [torch.empty(300, 264, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 264, dtype=torch.bfloat16, device="cuda")]
    plan.run(x, w, want[0], ws[0])
    plan.run(y, w, want[1], ws[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(o) for _ in range(20)] for o in want]
    for i in range(20):
        for j, z in enumerate((x, y)):
            plan.run(z, w, outs[j][i], ws[j], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(o, want[j]) for o in outs[j])
        plan.query_status(ws[j])


def test_one_workspace_for_all_calls_of_a_stream(agmm):
    """The products of several plans may share a workspace one after the other."""
    g = torch.Generator(device="cuda").manual_seed(6)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    a, b = agmm.LinearPlan(2056, 264, rhs_transpose=True), agmm.GatedPlan(520, 136)
    ws = a.new_workspace()
    assert a.workspace_bytes() == b.workspace_bytes()
    x, w, u, v = new(400, 2056), new(264, 2056), new(333, 520), new(520, 136)
    o, p = torch.empty(400, 264, dtype=torch.bfloat16, device="cuda"), torch.empty(333, 136, dtype=torch.bfloat16, device="cuda")
    a.run(x, w, o, ws)
    b.run(u, v, v, p, ws)
    want = o.clone(), p.clone()
    for _ in range(10):
        a.run(x, w, o.fill_(0), ws)
        b.run(u, v, v, p.fill_(0), ws)
        assert torch.equal(o, want[0]) and torch.equal(p, want[1])


def test_plans_made_while_capturing(agmm):
    """A plan asks the device for attributes only: it may be made inside a capture."""
    g = torch.Generator(device="cuda").manual_seed(7)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, y = new(40, 328), new(328, 152), new(40, 2056)
    want = agmm.gated_matmul(x, w, w, "gelu"), agmm.layer_norm(y)
    out, normed = torch.zeros_like(want[0]), torch.zeros_like(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = agmm.GatedPlan(328, 152, activation="gelu")
        ws = plan.new_workspace()
        plan.run(x, w, w, out, ws)
        norm = agmm.LayerNormPlan(2056)
        norm.run(y, normed)
    for _ in range(2):
        out.zero_()
        normed.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(normed, want[1])
