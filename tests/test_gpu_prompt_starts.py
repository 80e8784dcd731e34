"""Starts that fall, against the rules: what they stand for can be more work than is counted in 32 bits."""
import pytest
import torch

from attention_ref import attend, check, unit

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


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("times", [2048, 4097, 8200])
def test_more_work_than_is_counted(agmm, times):
    """2^20 rows, which overlap in memory, several times over: 2^19 items each time.  None is done."""
    rows = 2 ** 20
    plan = agmm.PromptPlan(128, 1, 64)
    ws = plan.new_workspace()
    q, out = (torch.full((8 * rows + 128 * 64,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k = torch.zeros((5, 1, 64), dtype=torch.bfloat16, device="cuda")
    starts = _ints([0, rows] * times)
    kv_starts = torch.zeros_like(starts)
    q_rows, out_rows = (x.as_strided((rows, 128, 64), (8, 64, 1)) for x in (q, out))
    for _ in range(2):
        plan.run(q_rows, k, k, starts, out_rows, ws, kv_starts=kv_starts)
        plan.query_status(ws)
    assert bool((out == 7).all())


@pytest.mark.parametrize("starts", [[300, 500, 100, 300], [600, 700] + [0, 20] * 15], ids=["few", "many"])
def test_starts_that_fall(agmm, starts):
    """A sequence whose end lies before its start is empty; the others are as they say."""
    hq, hk, d = 16, 4, 64
    g = torch.Generator().manual_seed(1)
    q, k, v = (unit(torch.randn((700, h, d), generator=g).bfloat16()) for h in (hq, hk, hk))
    plan = agmm.PromptPlan(hq, hk, d)
    ws, out = plan.new_workspace(), torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    plan.run(q.cuda(), k.cuda(), v.cuda(), _ints(starts), out, ws)
    plan.query_status(ws)
    out = out.cpu()
    told = torch.zeros(700, dtype=torch.bool)
    for a, b in zip(starts, starts[1:]):
        if b <= a:
            continue
        told[a:b] = True
        seen = torch.ones((b - a, b - a), dtype=torch.bool).tril()
        for h in range(hq):
            check(out[a:b, h], *attend(q[a:b, h], k[a:b, h // 4], v[a:b, h // 4], seen, d ** -0.5, q.dtype))
    assert bool((out[~told] == 7).all())
