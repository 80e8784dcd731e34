"""Attention of drafted tokens over a paged cache against the 64-bit form."""
import itertools

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


class Problem:
    """Random contexts and drafts in shuffled pages; unused places hold `poison`, unused table entries nonsense."""

    def __init__(self, ctx, nodes, hq, hk, d, page, dt, seed=0, poison=float("nan"), heads_first=False, std=1.5):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.nodes, self.hq, self.hk, self.d, self.page, self.dt = ctx, nodes, hq, hk, d, page, dt
        total = [c + n for c, n in zip(ctx, nodes)]
        need = [-(-t // page) for t in total]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g).tolist()
        shape = (pages, hk, page, d) if heads_first else (pages, page, hk, d)
        kc, vc = (torch.full(shape, poison, dtype=dt) for _ in range(2))
        self.kc, self.vc = (x.transpose(1, 2) if heads_first else x for x in (kc, vc))
        width = max(need + [1]) + 2
        nonsense = [-1, pages + 7, 2 ** 31 - 1, -2 ** 31]
        self.table, self.keys, self.values = [], [], []
        at = 0
        for t, m in zip(total, need):
            mine = order[at:at + m]
            at += m
            self.table.append(mine + [nonsense[i % 4] for i in range(width - m)])
            k = unit(torch.randn(t, hk, d, generator=g).to(dt))
            v = torch.randn(t, hk, d, generator=g).to(dt)
            for i in range(m):
                rows = slice(i * page, min(t, (i + 1) * page))
                n = rows.stop - rows.start
                self.kc[mine[i], :n], self.vc[mine[i], :n] = k[rows], v[rows]
            self.keys.append(k)
            self.values.append(v)
        self.starts = list(itertools.accumulate(nodes, initial=0))
        self.q = unit(torch.randn(sum(nodes), hq, d, generator=g).to(dt), std)

    def ref(self, seen_of, scale):
        """seen_of(s): [nodes, nodes] of booleans."""
        o = torch.zeros(self.q.shape, dtype=torch.float64)
        bound = torch.zeros_like(o)
        for s, (c, n) in enumerate(zip(self.ctx, self.nodes)):
            seen = torch.cat([torch.ones((n, c), dtype=torch.bool), seen_of(s)], 1)
            rows = slice(self.starts[s], self.starts[s] + n)
            for h in range(self.hq):
                hk = h * self.hk // self.hq
                o[rows, h], bound[rows, h] = attend(self.q[rows, h], self.keys[s][:, hk], self.values[s][:, hk], seen, scale, self.dt)
        return o, bound

    def run(self, agmm, mask=None, max_nodes=None, scale=None, stream=None):
        plan = agmm.TreePlan(self.hq, self.hk, self.d, page_size=self.page, max_nodes=max_nodes or max(self.nodes + [1]), scale=scale,
                             f16=self.dt == torch.float16)
        ws = plan.new_workspace()
        out = torch.full(self.q.shape, float("nan"), dtype=self.dt, device="cuda")
        self.plan, self.ws = plan, ws
        # a dense copy keeps the strides of heads-first caches
        kc, vc = self.kc.cuda(), self.vc.cuda()
        assert kc.stride() == self.kc.stride()
        plan.run(self.q.cuda(), kc, vc, _ints(self.table), _ints(self.ctx), _ints(self.starts), out, ws, mask=mask, stream=stream)
        plan.query_status(ws)
        return out.cpu()


def _chain(p):
    return lambda s: torch.ones((p.nodes[s], p.nodes[s]), dtype=torch.bool).tril()


def _random_parents(nodes, seed):
    g = torch.Generator().manual_seed(seed)
    return [[-1 if i == 0 else int(torch.randint(-1, i, (1,), generator=g)) for i in range(n)] for n in nodes]


def _seen(parents):
    def of(s):
        n = len(parents[s])
        m = torch.zeros((n, n), dtype=torch.bool)
        for i in range(n):
            j = i
            while j >= 0:
                m[i, j] = True
                j = parents[s][j]
        return m
    return of


@pytest.mark.parametrize("ctx", [[0], [1], [127, 128, 0], [129, 1000, 64, 255, 256]], ids=str)
@pytest.mark.parametrize("heads", [(8, 2, 128), (5, 1, 64), (2, 2, 128), (128, 1, 64), (14, 2, 128)], ids=str)
@pytest.mark.parametrize("page", [8, 16, 64, 128, 256])
def test_single_tokens(agmm, ctx, heads, page):
    hq, hk, d = heads
    dt = torch.bfloat16 if page != 16 else torch.float16
    p = Problem(ctx, [1] * len(ctx), hq, hk, d, page, dt, seed=page + len(ctx))
    want, bound = p.ref(_chain(p), d ** -0.5)
    check(p.run(agmm), want, bound)


@pytest.mark.parametrize("nodes", [[5, 1, 0, 7], [24, 24], [64, 3, 33], [130, 65, 2], [200]], ids=str)
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 1, 64), (3, 3, 64), (28, 4, 128)], ids=str)
@pytest.mark.parametrize("masked", [True, False])
def test_trees(agmm, nodes, heads, masked):
    hq, hk, d = heads
    ctx = [300, 0, 77, 129][:len(nodes)]
    dt = torch.float16 if d == 64 else torch.bfloat16
    p = Problem(ctx, nodes, hq, hk, d, 32, dt, seed=sum(nodes))
    parents = _random_parents(nodes, 5)
    want, bound = p.ref(_seen(parents) if masked else _chain(p), d ** -0.5)
    check(p.run(agmm, agmm.tree_mask(parents) if masked else None), want, bound)


@pytest.mark.parametrize("masked", [True, False])
def test_long_context_is_split_and_joined(agmm, masked):
    """One sequence much longer than the others: its keys are spread over the device and joined."""
    ctx, nodes = [20011, 3, 500], [6, 6, 6]
    p = Problem(ctx, nodes, 8, 2, 128, 64, torch.bfloat16, seed=1)
    parents = _random_parents(nodes, 2)
    want, bound = p.ref(_seen(parents) if masked else _chain(p), 0.1)
    got = p.run(agmm, agmm.tree_mask(parents) if masked else None, scale=0.1)
    check(got, want, bound)
    assert torch.equal(got, p.run(agmm, agmm.tree_mask(parents) if masked else None, scale=0.1)), "not the same bits twice"


def test_large_tree_over_a_long_context(agmm):
    """More rows than a pair of tiles holds, over split keys."""
    ctx, nodes = [5000, 900], [96, 40]
    p = Problem(ctx, nodes, 16, 2, 64, 16, torch.float16, seed=6)
    parents = _random_parents(nodes, 9)
    want, bound = p.ref(_seen(parents), 0.125)
    check(p.run(agmm, agmm.tree_mask(parents)), want, bound)


def test_any_mask_and_rows_that_see_nothing(agmm):
    """Masks that are no trees: some nodes see none, not even themselves; without a context their row is zero."""
    ctx, nodes = [0, 40, 0], [70, 70, 3]
    p = Problem(ctx, nodes, 4, 2, 64, 16, torch.bfloat16, seed=3)
    g = torch.Generator().manual_seed(0)
    seen = [torch.rand((n, n), generator=g) < 0.3 for n in nodes]
    for m in seen:
        m[1] = False
    seen[2][:] = False
    words = torch.zeros((sum(nodes), 2), dtype=torch.int64)
    for s, m in enumerate(seen):
        for i in range(nodes[s]):
            for w in range(2):
                bits = sum(1 << j for j in range(64) if 64 * w + j < nodes[s] and m[i, 64 * w + j])
                words[p.starts[s] + i, w] = bits - (1 << 64) if bits >> 63 else bits
    want, bound = p.ref(lambda s: seen[s], 0.125)
    got = p.run(agmm, words.cuda())
    check(got, want, bound)
    assert bool((got[1] == 0).all()) and bool((got[140:] == 0).all())
    # bits past a sequence's nodes are not looked at
    words[140:] = -1 << 3
    assert torch.equal(p.run(agmm, words.cuda()), got)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_node_reaches_only_those_that_see_it(agmm, value):
    """A drafted token whose key or value is not finite does not reach the nodes beside it."""
    for where in ("k", "v"):
        p = Problem([50], [9], 4, 2, 64, 16, torch.bfloat16, seed=8)
        parents = [[-1, 0, 0, 1, 1, 2, 2, 3, 5]]
        seen = _seen(parents)(0)
        want, bound = p.ref(lambda s: seen, 0.125)
        place = 50 + 2
        (p.kc if where == "k" else p.vc)[p.table[0][place // 16], place % 16, :, 7] = value
        got = p.run(agmm, agmm.tree_mask(parents))
        clear = ~seen[:, 2]
        check(got[clear], want[clear], bound[clear], where)
        if where == "v":
            assert not bool(torch.isfinite(got[~clear][..., 7]).any())
        elif value != value:
            assert bool(torch.isnan(got[~clear]).all())


def test_heads_first_caches(agmm):
    """Caches stored [pages, kv_heads, page_size, head_dim]."""
    p = Problem([200, 31], [3, 3], 8, 4, 128, 32, torch.bfloat16, seed=12, heads_first=True)
    want, bound = p.ref(_chain(p), 128 ** -0.5)
    check(p.run(agmm), want, bound)


def test_cache_past_32_bit_offsets(agmm):
    """Pages whose element offsets pass 2^31 and 2^32."""
    hk, page, d, dt = 8, 64, 128, torch.bfloat16
    pages = 2 ** 32 // (page * hk * d) + 9
    kc, vc = (torch.empty((pages, page, hk, d), dtype=dt, device="cuda") for _ in range(2))
    p = Problem([150], [2], 8, hk, d, page, dt, seed=4)
    far = [pages - 1, 2 ** 31 // (page * hk * d), pages // 2 + 5]
    for i in range(3):
        kc[far[i]], vc[far[i]] = p.kc[p.table[0][i]].cuda(), p.vc[p.table[0][i]].cuda()
    want, bound = p.ref(_chain(p), 0.1)
    out = agmm.tree_attention(p.q.cuda(), kc, vc, _ints([far]), _ints([150]), _ints([0, 2]), max_nodes=2, scale=0.1)
    check(out.cpu(), want, bound)


def test_lengths_and_pages_beyond_the_table_are_bounded(agmm):
    """A length past the page table counts what the table covers; a page outside the cache reads as zeros."""
    p = Problem([60], [1], 4, 2, 64, 16, torch.bfloat16, seed=10, poison=0.0)
    out = agmm.tree_attention(p.q.cuda(), p.kc.cuda(), p.vc.cuda(), _ints([p.table[0][:4]]), _ints([100000]), _ints([0, 1])).cpu()
    # 64 places: the 61 there are, and 3 of the last page's zeros
    zero = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    keys, values = torch.cat([p.keys[0], zero]), torch.cat([p.values[0], zero])
    for h in range(4):
        want, bound = attend(p.q[:, h], keys[:, h // 2], values[:, h // 2], torch.ones((1, 64), dtype=torch.bool), 0.125, p.dt)
        check(out[:, h], want, bound)
    outside = [p.table[0][:3] + [10 ** 6]]
    out = agmm.tree_attention(p.q.cuda(), p.kc.cuda(), p.vc.cuda(), _ints(outside), _ints([60]), _ints([0, 1])).cpu()
    zero = torch.zeros((13, 2, 64), dtype=torch.bfloat16)
    keys, values = torch.cat([p.keys[0][:48], zero]), torch.cat([p.values[0][:48], zero])
    for h in range(4):
        want, bound = attend(p.q[:, h], keys[:, h // 2], values[:, h // 2], torch.ones((1, 61), dtype=torch.bool), 0.125, p.dt)
        check(out[:, h], want, bound)


def test_nodes_past_the_bound_are_not_computed(agmm):
    p = Problem([40, 30], [5, 2], 4, 2, 64, 16, torch.bfloat16, seed=13)
    want, bound = p.ref(_chain(p), 0.125)
    got = p.run(agmm, max_nodes=3)
    assert bool(torch.isnan(got[3:5]).all())  # left as they were
    check(got[:3], want[:3], bound[:3])
    check(got[5:], want[5:], bound[5:])


def test_more_sequences_than_processors(agmm):
    g = torch.Generator().manual_seed(2)
    ctx = torch.randint(0, 300, (333,), generator=g).tolist()
    nodes = torch.randint(0, 3, (333,), generator=g).tolist()
    p = Problem(ctx, nodes, 4, 1, 64, 32, torch.float16, seed=14)
    want, bound = p.ref(_chain(p), 0.125)
    check(p.run(agmm), want, bound)


def test_stream_graph_and_workspace_reuse(agmm):
    p = Problem([3000, 10], [4, 4], 8, 2, 128, 64, torch.bfloat16, seed=15)
    first = p.run(agmm)
    args = [x.cuda() for x in (p.q, p.kc, p.vc)] + [_ints(p.table), _ints(p.ctx), _ints(p.starts)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = agmm.tree_attention(*args, max_nodes=4, stream=s)
    s.synchronize()
    assert torch.equal(out.cpu(), first)
    plan, ws = p.plan, p.ws
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(args[0])
    with torch.cuda.graph(graph):
        plan.run(*args, out, ws)
    args[2].neg_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), -first)
    # the same workspace, another shape of problem
    args[4].copy_(_ints([5, 10]))
    plan.run(*args, out, ws)
    plan.query_status(ws)
    args[4].copy_(_ints([3000, 10]))
    plan.run(*args, out, ws)
    plan.query_status(ws)
    assert torch.equal(out.cpu(), -first)


def test_nothing_to_do_and_refusals(agmm):
    new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    plan = agmm.TreePlan(4, 2, 64, page_size=16, max_nodes=70)
    ws = plan.new_workspace()
    q, out, kc = new(2, 4, 64), new(2, 4, 64), new(3, 16, 2, 64)
    table, ctx, starts = _ints([[0, 1], [2, 0]]), _ints([3, 4]), _ints([0, 1, 2])
    plan.run(q[:0], kc, kc, table, ctx, starts, out[:0], ws)
    plan.run(q, kc, kc, table, ctx, starts, out, ws)
    for bad in (
        lambda: plan.run(q[:, :2], kc, kc, table, ctx, starts, out, ws),
        lambda: plan.run(q.half(), kc, kc, table, ctx, starts, out, ws),
        lambda: plan.run(q, kc[:, :8], kc[:, :8], table, ctx, starts, out, ws),
        lambda: plan.run(q, kc, kc[:2], table, ctx, starts, out, ws),
        lambda: plan.run(q, kc, kc, table.long(), ctx, starts, out, ws),
        lambda: plan.run(q, kc, kc, table, ctx[:1], starts, out, ws),
        lambda: plan.run(q, kc, kc, table, ctx, starts[:2], out, ws),
        lambda: plan.run(q, kc, kc, table, ctx, starts, out[:1], ws),
        lambda: plan.run(q, kc, kc, table, ctx, starts, out, ws[:8]),
        lambda: plan.run(q, kc, kc, table, ctx, starts, out, ws, mask=new(2, 2, dtype=torch.int32)),
        lambda: plan.run(q, kc, kc, table, ctx, starts, out, ws, mask=new(1, 2, dtype=torch.int64)),
    ):
        with pytest.raises(ValueError):
            bad()
    status = lambda f: pytest.raises(agmm.AgmmError, f).value.status  # noqa: E731
    # 70 nodes need two words of mask
    assert status(lambda: plan.run(q, kc, kc, table, ctx, starts, out, ws, mask=new(2, 1, dtype=torch.int64))) == agmm.AGMM_ERR_INVALID_ARG
    assert status(lambda: agmm.TreePlan(4, 2, 64, page_size=48)) == agmm.AGMM_ERR_UNSUPPORTED
    assert status(lambda: agmm.TreePlan(4, 3, 64, page_size=16)) == agmm.AGMM_ERR_INVALID_ARG
    assert status(lambda: agmm.TreePlan(4, 2, 64, page_size=16, max_nodes=4000)) == agmm.AGMM_ERR_INVALID_ARG
