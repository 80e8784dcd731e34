"""A drafted token that sees one past the plan's bound: that one's key and value are in the cache."""
import pytest
import torch

from attention_ref import check
from test_gpu_tree import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nodes,bound", [(5, 3), (70, 40), (300, 130)])
def test_nodes_past_the_bound_are_seen(nodes, bound):
    import all_gather_gemm_agmm_gb300 as agmm
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    p = Problem([40, 9], [nodes, 2], 4, 2, 64, 16, torch.bfloat16, seed=nodes)
    seen = [torch.zeros((n, n), dtype=torch.bool) for n in p.nodes]
    seen[0].fill_diagonal_(True)
    seen[1].fill_diagonal_(True)
    words = -(-nodes // 64)
    seen[0][0, nodes - 1] = seen[0][2, bound] = True  # not among the first `bound`
    mask = torch.zeros((nodes + 2, words), dtype=torch.int64)
    for s, m in enumerate(seen):
        for i in range(m.shape[0]):
            for j in m[i].nonzero().flatten().tolist():
                v = int(mask[p.starts[s] + i, j // 64]) & (1 << 64) - 1 | 1 << j % 64
                mask[p.starts[s] + i, j // 64] = v - (1 << 64) if v >> 63 else v
    want, limit = p.ref(lambda s: seen[s], 0.125)
    got = p.run(agmm, mask.cuda(), max_nodes=bound)
    rows = list(range(bound)) + [nodes, nodes + 1]
    check(got[rows], want[rows], limit[rows])
    assert bool(torch.isnan(got[bound:nodes]).all())  # not computed: left as they were
