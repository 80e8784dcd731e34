"""Rows that are computed again for a hidden value that is not finite may take longer than a wait lasts."""
import pytest
import torch

from attention_ref import attend, check, unit

pytestmark = pytest.mark.gpu


def test_a_repair_outlasts_the_wait_limit(monkeypatch):
    """About 29 ms of repair with waits of 5 ms: the run is not given up, and its rows are right."""
    import all_gather_gemm_agmm_gb300 as agmm
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    n, heads, d, bad, dt = 4097, 32, 128, 4064, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(3)
    new = lambda h: torch.randn((n, h, d), generator=g, device="cuda").to(dt)  # noqa: E731
    q, k, v = unit(new(heads)), unit(new(1)), new(1)
    rows = torch.tensor([0, 100, 3967, 3968, 4000, 4063], device="cuda")
    seen = torch.arange(n, device="cuda")[None] <= rows[:, None]
    refs = [attend(q[rows, h], k[:, 0], v[:, 0], seen, d ** -0.5, dt) for h in range(0, heads, 5)]
    v[bad] = float("nan")
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    monkeypatch.setenv("AGMM_WAIT_LIMIT_MS", "5")
    plan = agmm.PromptPlan(heads, 1, d)
    monkeypatch.delenv("AGMM_WAIT_LIMIT_MS")
    ws, out = plan.new_workspace(), torch.empty_like(q)
    plan.run(q, k, v, starts, out, ws)
    assert plan.query_status(ws) == agmm.AGMM_OK
    for i, h in enumerate(range(0, heads, 5)):
        check(out[rows, h], *refs[i], f"head {h}")
    assert bool(torch.isnan(out[bad:]).all())
