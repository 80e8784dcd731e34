"""How many drafted tokens a sequence may have: given, or not."""
import pytest
import torch

from attention_ref import check
from test_gpu_tree import Problem, _chain, _ints, _random_parents, _seen

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


def _args(p):
    return [x.cuda() for x in (p.q, p.kc, p.vc)] + [_ints(p.table), _ints(p.ctx), _ints(p.starts)]


def _call(agmm, p, **kw):
    """tree_attention, whose output gets memory that held NaN."""
    args = _args(p)
    torch.cuda.synchronize()
    for n in range(4):
        torch.full(p.q.shape, float("nan"), dtype=p.dt, device="cuda")
    return agmm.tree_attention(*args, **kw).cpu()


@pytest.mark.parametrize("nodes", [[5, 2, 1], [0, 3, 0], [1, 1, 1], [17, 1, 15], [200, 0, 3]], ids=str)
@pytest.mark.parametrize("masked", [True, False])
def test_every_drafted_token_is_computed_by_default(agmm, nodes, masked):
    p = Problem([40, 300, 9], nodes, 8, 2, 64, 16, torch.bfloat16, seed=sum(nodes))
    parents = _random_parents(nodes, 3)
    want, bound = p.ref(_seen(parents) if masked else _chain(p), 0.125)
    check(_call(agmm, p, mask=agmm.tree_mask(parents) if masked else None), want, bound)


def test_a_mask_for_the_largest_tree_is_enough_by_default(agmm):
    """130 tokens in trees of 13: one word of mask each."""
    nodes = [13] * 10
    p = Problem([20 + i for i in range(10)], nodes, 4, 1, 64, 32, torch.float16, seed=1)
    parents = _random_parents(nodes, 4)
    mask = agmm.tree_mask(parents)
    assert mask.shape == (130, 1)
    want, bound = p.ref(_seen(parents), 0.125)
    check(_call(agmm, p, mask=mask), want, bound)


def test_a_large_batch_of_single_tokens_by_default(agmm):
    p = Problem([i % 70 for i in range(1100)], [1] * 1100, 1, 1, 64, 16, torch.bfloat16, seed=2)
    want, bound = p.ref(_chain(p), 0.125)
    check(_call(agmm, p), want, bound)


def test_more_tokens_than_the_given_bound_allows(agmm):
    p = Problem([40, 30], [5, 2], 4, 2, 64, 16, torch.bfloat16, seed=5)
    with pytest.raises(ValueError):
        _call(agmm, p, max_nodes=3)
    # a bound that only one of them passes cannot be seen on the host: its rows are zero
    p = Problem([40, 30], [5, 1], 4, 2, 64, 16, torch.bfloat16, seed=6)
    want, bound = p.ref(_chain(p), 0.125)
    got = _call(agmm, p, max_nodes=3)
    check(got[:3], want[:3], bound[:3])
    check(got[5:], want[5:], bound[5:])
    assert bool((got[3:5] == 0).all())


def test_a_workspace_for_fewer_nodes(agmm):
    """A plan's workspace goes with the plan's bound; without the bound the function says so."""
    p = Problem([40] * 32, [1] * 32, 8, 2, 64, 16, torch.bfloat16, seed=7)
    want, bound = p.ref(_chain(p), 0.125)
    ws = agmm.TreePlan(8, 2, 64, page_size=16, max_nodes=1).new_workspace()
    check(_call(agmm, p, max_nodes=1, workspace=ws), want, bound)
    with pytest.raises(ValueError, match="max_nodes"):
        _call(agmm, p, workspace=ws)
    ws = agmm.TreePlan(8, 2, 64, page_size=16, max_nodes=32).new_workspace()
    check(_call(agmm, p, workspace=ws), want, bound)
