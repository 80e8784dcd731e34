"""Attention of packed prompts against the 64-bit form."""
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


def _edges(lens):
    return list(itertools.accumulate(lens, initial=0))


def _make(lens, kv_lens, hq, hk, d, dt, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    q = unit(torch.randn(sum(lens), hq, d, generator=g).to(dt), std)
    k = unit(torch.randn(sum(kv_lens), hk, d, generator=g).to(dt))
    v = torch.randn(sum(kv_lens), hk, d, generator=g).to(dt)
    return q, k, v


def _ref(q, k, v, lens, kv_lens, causal, scale):
    hq, hk = q.shape[1], k.shape[1]
    o, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    at, kv_at = _edges(lens), _edges(kv_lens)
    for s, (n, m) in enumerate(zip(lens, kv_lens)):
        seen = torch.ones((n, m), dtype=torch.bool)
        if causal:
            seen = seen.tril(m - n)
        rows, cols = slice(at[s], at[s] + n), slice(kv_at[s], kv_at[s] + m)
        for h in range(hq):
            o[rows, h], bound[rows, h] = attend(q[rows, h], k[cols, h * hk // hq], v[cols, h * hk // hq], seen, scale, q.dtype)
    return o, bound


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


LENS = [
    [1],
    [2, 1, 127, 128, 129],
    [0, 300, 0, 257, 0],
    [255, 256, 257],
    [513, 3, 700],
]


@pytest.mark.parametrize("lens", LENS, ids=["-".join(map(str, x)) for x in LENS])
@pytest.mark.parametrize("heads", [(8, 2, 128), (5, 1, 64), (3, 3, 128), (16, 2, 64)], ids=str)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_causal(agmm, lens, heads, dt):
    hq, hk, d = heads
    q, k, v = _make(lens, lens, hq, hk, d, dt, seed=sum(lens))
    want, bound = _ref(q, k, v, lens, lens, True, d ** -0.5)
    out = torch.full(q.shape, float("nan"), dtype=dt, device="cuda")
    plan = agmm.PromptPlan(hq, hk, d, f16=dt == torch.float16)
    ws = plan.new_workspace()
    plan.run(q.cuda(), k.cuda(), v.cuda(), _ints(_edges(lens)), out, ws)
    plan.query_status(ws)
    check(out.cpu(), want, bound)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,kv_lens", [([1, 40, 300], [1000, 41, 300]), ([130, 7, 5], [64, 0, 700]),
                                          ([260, 1, 128], [131, 129, 1]), ([5], [2049])], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_other_key_lengths(agmm, causal, lens, kv_lens, d):
    """Keys before the queries (the piece of a prompt behind a prefix), and fewer keys than queries: rows that see nothing are zero."""
    dt = torch.bfloat16
    q, k, v = _make(lens, kv_lens, 8, 4, d, dt, seed=7)
    want, bound = _ref(q, k, v, lens, kv_lens, causal, 0.11)
    out = torch.full(q.shape, float("nan"), dtype=dt, device="cuda")
    agmm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _ints(_edges(lens)), _ints(_edges(kv_lens)), scale=0.11, causal=causal, out=out)
    check(out.cpu(), want, bound)


def test_long_prompt_on_some_rows(agmm):
    """6000 tokens: many key tiles, the maximum moving over them; every 37th row and the last are compared."""
    dt, n, d = torch.bfloat16, 6001, 128
    q, k, v = _make([n], [n], 2, 1, d, dt, seed=2, std=4.0)
    k = (k.float() * torch.linspace(0.2, 2.0, n)[:, None, None]).to(dt)  # later keys score higher and higher
    out = agmm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _ints([0, n])).cpu()
    rows = torch.cat([torch.arange(0, n, 37), torch.tensor([n - 1])])
    seen = torch.arange(n)[None] <= rows[:, None]
    for h in range(2):
        want, bound = attend(q[rows, h], k[:, 0], v[:, 0], seen, d ** -0.5, dt)
        # scores here reach 4 * 2 * sqrt(d): their float32 error is 8 times the usual
        check(out[rows, h], want, bound + 8 * 5e-4 * (bound / (2.0 ** -8 + 5e-4)))


def test_large_scores(agmm):
    """Scores of thousands: the weights are all but one-hot, and no exponential overflows."""
    for dt in (torch.bfloat16, torch.float16):
        lens, d = [200], 64
        q, k, v = _make(lens, lens, 2, 2, d, dt, seed=11, std=60.0)
        k = (k.float() * 8).to(dt)
        out = agmm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _ints([0, 200]), scale=1.0).cpu()
        assert bool(torch.isfinite(out).all())
        s = torch.einsum("qhd,khd->hqk", q.double(), k.double()).masked_fill(~torch.ones(200, 200, dtype=torch.bool).tril(), -1e300)
        top, second = s.topk(2, -1).values.unbind(-1)
        sure = top - second > 40  # other weights are below e^-40
        best = v[s.argmax(-1).T, torch.arange(2)[None]]
        assert torch.equal(out[sure.T], best[sure.T])


def test_what_lies_outside_is_not_used(agmm):
    """NaN and infinities in the rows of no sequence and past the ends do not reach an output; rows of no sequence are not written."""
    dt, d, hq, hk = torch.bfloat16, 128, 4, 2
    lens = [130, 70]
    q, k, v = _make(lens, lens, hq, hk, d, dt, seed=5)
    want, bound = _ref(q, k, v, lens, lens, True, d ** -0.5)
    lead, gap = 9, 100
    starts = _ints([lead, lead + 130, lead + 200])
    buf = torch.full((lead + 200 + gap, hq + 2 * hk, d), float("nan"), dtype=dt, device="cuda")
    buf[-3:] = float("inf")
    rows = buf[lead:lead + 200]
    rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:] = q.cuda(), k.cuda(), v.cuda()
    out = torch.full((lead + 200 + gap, hq, d), 5.0, dtype=dt, device="cuda")
    plan = agmm.PromptPlan(hq, hk, d)
    plan.run(buf[:, :hq], buf[:, hq:hq + hk], buf[:, hq + hk:], starts, out, plan.new_workspace())
    check(out[lead:lead + 200].cpu(), want, bound)
    assert bool((out[:lead] == 5).all()) and bool((out[lead + 200:] == 5).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_later_tokens_do_not_reach_earlier_rows(agmm, value, where):
    """A value that is not finite in a key or value row reaches the rows that see it, and no earlier one of its tile."""
    dt, d, n, bad = torch.float16, 64, 300, (70, 200)
    q, k, v = _make([n], [n], 4, 2, d, dt, seed=15)
    want, bound = _ref(q, k, v, [n], [n], True, d ** -0.5)
    for b in bad:
        (k if where == "k" else v)[b, 0, 3] = value
    out = agmm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _ints([0, n])).cpu()
    check(out[:, 2:], want[:, 2:], bound[:, 2:], "the other key head")
    check(out[:bad[0], :2], want[:bad[0], :2], bound[:bad[0], :2], "rows before")
    if where == "v":
        col = out[bad[0]:, :2, 3]
        assert not bool(torch.isfinite(col).any())
        rest = [c for c in range(d) if c != 3]
        check(out[bad[0]:, :2, rest], want[bad[0]:, :2, rest], bound[bad[0]:, :2, rest], "other columns")
        if value > 0:  # +inf stays +inf
            assert bool((col == value).all())
    elif value != value:
        assert bool(torch.isnan(out[bad[0]:, :2]).all())


def test_strides(agmm):
    """Heads before tokens, and heads taken from wider rows."""
    dt, d, hq, hk, lens = torch.bfloat16, 64, 6, 3, [150, 31]
    q, k, v = _make(lens, lens, hq, hk, d, dt, seed=9)
    want, bound = _ref(q, k, v, lens, lens, True, d ** -0.5)
    q2 = q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    k2 = torch.zeros(181, 2 * hk, 2 * d, dtype=dt, device="cuda")[:, ::2, :d]
    k2.copy_(k)
    v2 = v.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros(hq, 181, d + 8, dtype=dt, device="cuda").transpose(0, 1)[..., :d]
    agmm.prompt_attention(q2, k2, v2, _ints(_edges(lens)), out=out)
    check(out.cpu(), want, bound)


def test_many_sequences(agmm):
    """More sequences than a warp scans at once, most of them tiny."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 6, (333,), generator=g).tolist() + [140] + torch.randint(0, 9, (70,), generator=g).tolist()
    dt, d = torch.float16, 64
    q, k, v = _make(lens, lens, 2, 1, d, dt, seed=3)
    want, bound = _ref(q, k, v, lens, lens, True, d ** -0.5)
    out = agmm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _ints(_edges(lens)))
    check(out.cpu(), want, bound)


@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 2, 64)], ids=str)
def test_many_items_of_all_sizes(agmm, heads):
    """Enough items that they are drawn, of many lengths: one and two tiles to a set, two heads to an item and one."""
    hq, hk, d = heads
    g = torch.Generator().manual_seed(hq)
    lens = torch.randint(0, 280, (50,), generator=g).tolist() + [600, 1, 128, 129, 385, 384, 256, 0, 511]
    kv_lens = [n + int(torch.randint(0, 200, (1,), generator=g)) for n in lens]
    q, k, v = _make(lens, kv_lens, hq, hk, d, torch.bfloat16, seed=21)
    want, bound = _ref(q, k, v, lens, kv_lens, True, d ** -0.5)
    plan = agmm.PromptPlan(hq, hk, d)
    ws = plan.new_workspace()
    for _ in range(2):
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
        plan.run(q.cuda(), k.cuda(), v.cuda(), _ints(_edges(lens)), out, ws, kv_starts=_ints(_edges(kv_lens)))
        plan.query_status(ws)
        check(out.cpu(), want, bound)


def test_hidden_values_in_a_cut_prompt(agmm):
    """A prompt that is cut along its keys, with values that are not finite near its end: earlier rows are as they were."""
    dt, d, n = torch.bfloat16, 128, 3001
    q, k, v = _make([n], [n], 2, 1, d, dt, seed=23)
    rows = torch.tensor([0, 100, 1500, 2816, 2900, 2949, 2950, 2999, 3000])
    seen = torch.arange(n)[None] <= rows[:, None]
    refs = [attend(q[rows, h], k[:, 0], v[:, 0], seen, d ** -0.5, dt) for h in range(2)]
    v[2950, 0, 7] = float("inf")
    v[3000, 0, 9] = float("nan")
    out = agmm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), _ints([0, n])).cpu()[rows]
    for h in range(2):
        want, bound = refs[h]
        clear = [c for c in range(d) if c not in (7, 9)]
        check(out[:, h][:, clear], want[:, clear], bound[:, clear], "other columns")
        check(out[:6, h], want[:6], bound[:6], "rows before")
        assert bool((out[6:, h, 7] == float("inf")).all())
        check(out[6:8, h, 9:10], want[6:8, 9:10], bound[6:8, 9:10])
        assert bool(torch.isnan(out[8, h, 9]))


def test_same_bits_every_time_and_on_another_stream(agmm):
    dt, d, lens = torch.bfloat16, 128, [700, 90, 1100]
    q, k, v = (x.cuda() for x in _make(lens, lens, 8, 2, d, dt, seed=4))
    starts = _ints(_edges(lens))
    plan = agmm.PromptPlan(8, 2, d)
    ws = plan.new_workspace()
    first = torch.empty_like(q)
    plan.run(q, k, v, starts, first, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        out = agmm.prompt_attention(q, k, v, starts, stream=s)
        s.synchronize()
        assert torch.equal(out, first)
    # a captured run, replayed on new values in the same buffers
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        plan.run(q, k, v, starts, out, ws)
    v.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -first)
    plan.query_status(ws)


def test_nothing_to_do(agmm):
    e = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert agmm.prompt_attention(e, e[:, :2], e[:, :2], _ints([0])).shape == (0, 4, 64)
    q = torch.ones((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    out = agmm.prompt_attention(q, e[:, :2], e[:, :2], _ints([0, 3]), _ints([0, 0]))  # queries, and no key at all
    assert bool((out == 0).all())


def test_refusals(agmm):
    dt = torch.bfloat16
    new = lambda *s, dtype=dt: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    plan = agmm.PromptPlan(4, 2, 64)
    ws = plan.new_workspace()
    q, k, out, starts = new(5, 4, 64), new(5, 2, 64), new(5, 4, 64), _ints([0, 5])
    plan.run(q, k, k, starts, out, ws)
    for bad in (
        lambda: plan.run(q[:, :2], k, k, starts, out, ws),
        lambda: plan.run(q.float(), k, k, starts, out, ws),
        lambda: plan.run(q.cpu(), k, k, starts, out, ws),
        lambda: plan.run(q, k[:3], k, starts, out, ws),
        lambda: plan.run(q, k[:3], k[:3], starts, out, ws),           # other rows need kv_starts
        lambda: plan.run(q, k, k, starts.long(), out, ws),
        lambda: plan.run(q, k, k, starts, out[:4], ws),
        lambda: plan.run(q, k, k, starts, out, ws, kv_starts=_ints([0, 2, 5])),
        lambda: plan.run(q, k, k, starts, out, ws[:16]),
        lambda: plan.run(q, k.transpose(1, 2).contiguous().transpose(1, 2), k, starts, out, ws),
    ):
        with pytest.raises(ValueError):
            bad()
    odd = new(5, 4, 68)[..., :64]  # strides of 4 elements' grain
    assert pytest.raises(agmm.AgmmError, lambda: plan.run(odd, k, k, starts, out, ws)).value.status == agmm.AGMM_ERR_ALIGNMENT
