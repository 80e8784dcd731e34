"""Rows and places past what 32-bit counters hold are refused (the kernels look a little past every end)."""
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


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _status(agmm, f):
    return pytest.raises(agmm.AgmmError, f).value.status


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 1000, 2 ** 31 - 4096])
def test_rows_of_keys(agmm, rows):
    """Rows that share their memory: nothing is launched."""
    plan = agmm.PromptPlan(2, 1, 64)
    ws = plan.new_workspace()
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda").expand(rows, 1, 64)
    out = torch.full_like(q, 7.0)
    run = lambda: plan.run(q, k, k, _ints([0, 3]), out, ws, kv_starts=_ints([0, 5]))  # noqa: E731
    assert _status(agmm, run) == agmm.AGMM_ERR_INVALID_ARG
    assert bool((out == 7).all())


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 4096])
def test_rows_of_queries(agmm, rows):
    plan = agmm.PromptPlan(2, 1, 64)
    ws = plan.new_workspace()
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda").expand(rows, 2, 64)
    k = torch.zeros((5, 1, 64), dtype=torch.bfloat16, device="cuda")
    run = lambda: plan.run(q, k, k, _ints([0, 3]), q, ws, kv_starts=_ints([0, 5]))  # noqa: E731
    assert _status(agmm, run) == agmm.AGMM_ERR_INVALID_ARG


@pytest.mark.parametrize("page", [8, 256])
def test_places_of_a_page_table(agmm, page):
    plan = agmm.TreePlan(2, 1, 64, page_size=page, max_nodes=3)
    ws = plan.new_workspace()
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((2, page, 1, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    most = (2 ** 31 - 4097) // page
    for pages in (2 ** 31 // page - 1, most + 1):
        table = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
        run = lambda: plan.run(q, kc, kc, table, _ints([4]), _ints([0, 3]), out, ws)  # noqa: E731
        assert _status(agmm, run) == agmm.AGMM_ERR_INVALID_ARG
    assert bool((out == 7).all())
    # the widest table: a short context in it is as any other
    plan.run(q, kc, kc, table[:, :most], _ints([4]), _ints([0, 3]), out, ws)
    plan.query_status(ws)
    assert bool((out == 0).all())
