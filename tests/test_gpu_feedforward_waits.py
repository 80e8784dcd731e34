"""The bounds of the feed-forward products' waits count from the end of the kernel before: a
launch may be resident long before that, and its inputs are not there until then."""
import pytest
import torch

pytestmark = pytest.mark.gpu
LONG = 1 << 20  # values to a row of the kernel before: 256 MB of weights through one CTA, about 3 ms


@pytest.fixture(scope="module")
def agmm():
    import all_gather_gemm_agmm_gb300 as m
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    m.load_library()
    return m


@pytest.fixture(scope="module")
def long_call(agmm):
    """A product of one CTA, which leaves the other SMs to the launch behind it."""
    with pytest.MonkeyPatch.context() as env:
        env.setenv("AGMM_PATH", "1")
        env.setenv("AGMM_SPLITK", "1")
        plan = agmm.LinearPlan(LONG, 128, rhs_transpose=True)
    x, w = (torch.zeros(n, LONG, dtype=torch.bfloat16, device="cuda") for n in (1, 128))
    out, ws = torch.empty(1, 128, dtype=torch.bfloat16, device="cuda"), plan.new_workspace()
    yield lambda: plan.run(x, w, out, ws)
    plan.query_status(ws)


@pytest.mark.parametrize("rows, env", [(1, {"AGMM_SPLITK": "1"}), (40, {"AGMM_SPLITK": "4"}), (300, {}), (300, {"AGMM_STREAMK": "1"})],
                         ids=["swapped", "split", "rows", "cut"])
def test_a_long_kernel_before(agmm, long_call, monkeypatch, rows, env):
    g = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, d, r = new(rows, 1032), new(264, 1032), new(rows, 264), new(rows, 264)
    for k, v in env.items():
        monkeypatch.setenv(k, v)
    monkeypatch.setenv("AGMM_WAIT_LIMIT_MS", "1")
    plan = agmm.LinearPlan(1032, 264, rhs_transpose=True)
    ws = plan.new_workspace()

    def step():
        out, dx, dw = torch.zeros_like(d), torch.zeros_like(x), torch.zeros_like(w)
        return (out, dx, dw), (lambda: plan.run(x, w, out, ws, residual=r), lambda: plan.backward(d, x, w, ws, dx=dx, dw=dw))

    want, calls = step()
    for call in calls:
        call()
    assert plan.query_status(ws) == agmm.AGMM_OK
    got, calls = step()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for call in calls:
        torch.cuda.synchronize()
        begin.record()
        long_call()
        end.record()
        torch.cuda.synchronize()
        assert begin.elapsed_time(end) > 2, "the kernel before has to outlast the limit"
        long_call()
        call()
    assert plan.query_status(ws) == agmm.AGMM_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)
