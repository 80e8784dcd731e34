"""A device-side wait of the feed-forward products that runs out is reported, and the context
and the workspace stay usable.

The test hook AGMM_TEST_DROP_ARRIVE makes each producer skip its first load, so the wait for it
runs out (here after 200 ms): the kernel records AGMM_ERR_TIMEOUT, every role leaves its loop,
copies and products in flight end, tensor memory is freed and the kernel returns."""
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


@pytest.mark.parametrize("rows,env", [(5, {"AGMM_SPLITK": "1"}), (5, {"AGMM_SPLITK": "4"}), (300, {"AGMM_STREAMK": "0"}),
                                      (300, {"AGMM_STREAMK": "1"}), (300, {"AGMM_BN": "128", "AGMM_SPLITK": "3"})],
                         ids=["swapped", "split", "rows", "cut", "pairs"])
def test_dropped_load_times_out_and_recovers(agmm, rows, env, monkeypatch):
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w = new(rows, 1032), new(264, 1032)
    for k, v in env.items():
        monkeypatch.setenv(k, v)
    make = lambda: agmm.GatedPlan(1032, 264, rhs_transpose=True)  # noqa: E731
    good = make()
    ws = good.new_workspace()
    want, out = (torch.empty(rows, 264, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    good.run(x, w, w, want, ws)
    assert good.query_status(ws) == agmm.AGMM_OK

    monkeypatch.setenv("AGMM_TEST_DROP_ARRIVE", "1")
    monkeypatch.setenv("AGMM_WAIT_LIMIT_MS", "200")
    bad = make()
    bad_ws = bad.new_workspace()
    bad.run(x, w, w, out, bad_ws)
    with pytest.raises(agmm.AgmmError) as err:
        bad.query_status(bad_ws)
    assert err.value.status == agmm.AGMM_ERR_TIMEOUT and "ran out" in str(err.value)
    assert bad.query_status(bad_ws) == agmm.AGMM_OK  # cleared by the query
    torch.cuda.synchronize()

    good.run(x, w, w, out, bad_ws)  # the workspace, too
    assert good.query_status(bad_ws) == agmm.AGMM_OK
    assert torch.equal(out, want)
