"""A device-side wait that runs out is reported, and the context stays usable.

The test hook AGMM_TEST_DROP_ARRIVE makes the producer skip its first load, so
the wait for it runs out (here after 200 ms): the kernel records
AGMM_ERR_TIMEOUT, every role leaves its loop, copies and products in flight end,
tensor memory is freed and the kernel returns.  Nothing traps or touches an
invalid address."""
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


@pytest.mark.parametrize("kind", ["prompt", "tree"])
@pytest.mark.parametrize("d", [64, 128])
def test_dropped_load_times_out_and_recovers(agmm, kind, d, monkeypatch):
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def make():
        return agmm.PromptPlan(4, 2, d) if kind == "prompt" else agmm.TreePlan(4, 2, d, page_size=64, max_nodes=2)

    if kind == "prompt":
        q, k, v = new(700, 4, d), new(700, 2, d), new(700, 2, d)
        run = lambda plan, out, ws: plan.run(q, k, v, ints([0, 300, 700]), out, ws)  # noqa: E731
    else:
        q, k, v = new(4, 4, d), new(40, 64, 2, d), new(40, 64, 2, d)
        table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
        run = lambda plan, out, ws: plan.run(q, k, v, table, ints([1200, 7]), ints([0, 2, 4]), out, ws)  # noqa: E731

    good = make()
    ws = good.new_workspace()
    want, out = torch.empty_like(q), torch.empty_like(q)
    run(good, want, ws)
    assert good.query_status(ws) == agmm.AGMM_OK

    monkeypatch.setenv("AGMM_TEST_DROP_ARRIVE", "1")
    monkeypatch.setenv("AGMM_WAIT_LIMIT_MS", "200")
    bad = make()
    monkeypatch.delenv("AGMM_TEST_DROP_ARRIVE")
    monkeypatch.delenv("AGMM_WAIT_LIMIT_MS")
    bad_ws = bad.new_workspace()
    run(bad, out, bad_ws)
    with pytest.raises(agmm.AgmmError) as err:
        bad.query_status(bad_ws)
    assert err.value.status == agmm.AGMM_ERR_TIMEOUT and "ran out" in str(err.value)
    assert bad.query_status(bad_ws) == agmm.AGMM_OK  # cleared by the query

    run(good, out, ws)
    assert good.query_status(ws) == agmm.AGMM_OK
    assert torch.equal(out, want)
