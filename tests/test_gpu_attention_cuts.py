"""Every key counts once, also at the edges of tiles and of the parts that work is cut into.

Queries of zero give n keys equal weights, which are exact in any format: a value of 1 in a
column of its own for each of 128 keys at a time makes that column 1 / n, to the rounding of
1 / n (float32) and of the output: 2^-8 of it in bf16 and 2^-11 in fp16."""
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


def _check(out, keys, first, dt):
    """out [rows, heads, d]: column j is 1 / keys[row] where the row sees key first + j, else 0."""
    d = out.shape[2]
    at = first + torch.arange(d, device="cuda")
    want = torch.where(at[None] < keys[:, None], 1.0 / keys[:, None].double(), 0.0)[:, None].expand(out.shape)
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dt]
    off = (out.double() - want).abs() > u * want + (2.0 ** -25 if dt == torch.float16 else 0)
    assert not bool(off.any()), f"keys {first}..{first + d - 1}: {off.nonzero()[:5].tolist()} are wrong"


@pytest.mark.parametrize("d,dt", [(128, torch.bfloat16), (64, torch.float16)], ids=["128-bf16", "64-f16"])
@pytest.mark.parametrize("contexts,nodes", [([20011, 3, 500], 6), ([1000], 1), ([4097, 128, 127, 129, 0, 2900], 1), ([7000, 900], 40)],
                         ids=str)
def test_trees(agmm, d, dt, contexts, nodes):
    page, hq, hk = 32, 8, 2
    need = [-(-(c + nodes) // page) for c in contexts]
    pages = sum(need)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(pages)).split(need)
    table = torch.zeros((len(contexts), max(need)), dtype=torch.int32)
    for s, mine in enumerate(order):
        table[s, :len(mine)] = mine
    kc, vc = (torch.zeros((pages, page, hk, d), dtype=dt, device="cuda") for _ in range(2))
    q = torch.zeros((nodes * len(contexts), hq, d), dtype=dt, device="cuda")
    plan = agmm.TreePlan(hq, hk, d, page_size=page, max_nodes=nodes, f16=dt == torch.float16)
    ws, out = plan.new_workspace(), torch.empty_like(q)
    args = table.cuda(), _ints(contexts), _ints([nodes * s for s in range(len(contexts) + 1)])
    keys = torch.cat([c + 1 + torch.arange(nodes) for c in contexts]).cuda()
    flat = vc.view(-1, hk, d)
    for first in range(0, max(contexts) + nodes, d):
        vc.zero_()
        for s, mine in enumerate(order):
            place = torch.arange(first, max(first, min(first + d, contexts[s] + nodes)))
            if len(place):
                flat[(mine[place // page] * page + place % page).cuda(), :, torch.arange(len(place), device="cuda")] = 1.0
        plan.run(q, kc, vc, *args, out, ws)
        _check(out, keys, first, dt)
    plan.query_status(ws)


@pytest.mark.parametrize("d,dt", [(128, torch.float16), (64, torch.bfloat16)], ids=["128-f16", "64-bf16"])
@pytest.mark.parametrize("lens,prefixes", [([5], [19990]), ([300, 129], [2000, 1500]), ([3000], [0]), ([40] * 40, [100] * 40)], ids=str)
def test_prompts(agmm, d, dt, lens, prefixes):
    """Cut along the keys, and (the last case) drawn whole."""
    hq, hk = 8, 4
    kv = [n + p for n, p in zip(lens, prefixes)]
    kv_at = [sum(kv[:i]) for i in range(len(kv) + 1)]
    q = torch.zeros((sum(lens), hq, d), dtype=dt, device="cuda")
    k, v = (torch.zeros((sum(kv), hk, d), dtype=dt, device="cuda") for _ in range(2))
    plan = agmm.PromptPlan(hq, hk, d, f16=dt == torch.float16)
    ws, out = plan.new_workspace(), torch.empty_like(q)
    starts, kv_starts = _ints([sum(lens[:i]) for i in range(len(lens) + 1)]), _ints(kv_at)
    keys = torch.cat([p + 1 + torch.arange(n) for n, p in zip(lens, prefixes)]).cuda()
    for first in range(0, max(kv), d):
        v.zero_()
        for s, m in enumerate(kv):
            place = torch.arange(first, max(first, min(first + d, m)), device="cuda")
            if len(place):
                v[kv_at[s] + place, :, place - first] = 1.0
        plan.run(q, k, v, starts, out, ws, kv_starts=kv_starts)
        _check(out, keys, first, dt)
    plan.query_status(ws)
