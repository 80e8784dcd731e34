"""A workspace whose run has timed out, asked about, works again."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_drawn_items_after_a_timeout(monkeypatch):
    """Prompts with so many items that they are drawn from a counter in the workspace; the run that
    times out leaves it somewhere in between."""
    import all_gather_gemm_agmm_gb300 as agmm
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = [300, 20, 129, 1] * 8
    starts = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    new = lambda h: torch.randn((sum(lens), h, 64), generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v = new(32), new(8), new(8)
    good = agmm.PromptPlan(32, 8, 64)
    want = torch.empty_like(q)
    ws = good.new_workspace()
    good.run(q, k, v, starts, want, ws)
    assert good.query_status(ws) == agmm.AGMM_OK

    monkeypatch.setenv("AGMM_TEST_DROP_ARRIVE", "1")
    monkeypatch.setenv("AGMM_WAIT_LIMIT_MS", "200")
    bad = agmm.PromptPlan(32, 8, 64)
    monkeypatch.delenv("AGMM_TEST_DROP_ARRIVE")
    monkeypatch.delenv("AGMM_WAIT_LIMIT_MS")
    ws = bad.new_workspace()
    out = torch.empty_like(q)
    bad.run(q, k, v, starts, out, ws)
    with pytest.raises(agmm.AgmmError) as err:
        bad.query_status(ws)
    assert err.value.status == agmm.AGMM_ERR_TIMEOUT
    for _ in range(2):
        out.fill_(float("nan"))
        good.run(q, k, v, starts, out, ws)
        assert good.query_status(ws) == agmm.AGMM_OK
        assert torch.equal(out, want)
