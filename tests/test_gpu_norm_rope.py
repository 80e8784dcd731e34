"""Norms with rotation and cache writes against the 64-bit form."""
import pytest
import torch

from attention_ref import check, rope_ref

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


CASES = [
    # tokens, q heads, kv heads, d, rotary, sections, interleaved, adjacent, dtype, weights
    (1, 32, 8, 128, 128, None, False, False, torch.bfloat16, True),
    (3, 5, 1, 64, 64, None, False, False, torch.float16, True),
    (77, 16, 2, 64, 64, (8, 12, 12), False, False, torch.bfloat16, True),
    (130, 28, 4, 128, 128, (24, 20, 20), True, False, torch.float16, True),
    (9, 7, 7, 128, 64, (20, 12), False, False, torch.bfloat16, True),       # part of the head rotates
    (11, 40, 8, 128, 128, (16, 16, 16, 16), False, True, torch.bfloat16, True),  # adjacent pairs
    (5, 3, 3, 256, 48, (24,), False, True, torch.float16, True),
    (6, 6, 2, 256, 256, None, False, False, torch.bfloat16, False),          # no norm
    (4, 2, 1, 64, 0, (), False, False, torch.float16, True),                 # no rotation
    (2, 130, 2, 64, 64, None, False, False, torch.bfloat16, True),           # more heads than a block holds at once
]


def _inputs(case, seed, dev="cuda"):
    t, hq, hk, d, rot, sections, inter, adj, dt, weights = case
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(t, hq + 2 * hk, d, generator=g) * 2).to(dt)
    wq = (1 + 0.3 * torch.randn(d, generator=g)).to(dt) if weights else None
    wk = (1 + 0.3 * torch.randn(d, generator=g)).to(dt) if weights else None
    axes = 1 if sections is None else max(1, len(sections))
    pos = torch.randint(-5, 1 << 20, (axes, t), generator=g)
    return qkv, wq, wk, pos


def _ref(agmm, case, qkv, wq, wk, pos, eps=1e-6, base=1e6):
    t, hq, hk, d, rot, sections, inter, adj, dt, weights = case
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    axis = agmm.rotary_axes((rot // 2,) if sections is None else sections, inter)
    return rope_ref(qkv, wq, wk, pos, freq, axis, rot, adj, eps, hq, hk)


def _plan(agmm, case):
    t, hq, hk, d, rot, sections, inter, adj, dt, weights = case
    return agmm.NormRopePlan(hq, hk, d, rotary_dim=rot, sections=sections or ((0,) if sections == () else None),
                             interleaved=inter, adjacent=adj, base=1e6, f16=dt == torch.float16)


@pytest.mark.parametrize("case", CASES, ids=[f"t{c[0]}_h{c[1]}-{c[2]}_d{c[3]}_r{c[4]}" for c in CASES])
@pytest.mark.parametrize("form", ["packed", "cache", "in_place"])
def test_against_the_formula(agmm, case, form):
    t, hq, hk, d, rot, sections, inter, adj, dt, weights = case
    qkv, wq, wk, pos = _inputs(case, 3)
    q_ref, k_ref, v_ref, bq, bk = _ref(agmm, case, qkv, wq, wk, pos)
    plan = _plan(agmm, case)
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    rows = qkv.cuda()
    positions = pos.cuda() if form == "cache" else pos.int().cuda()
    if form == "in_place":
        # the rows lie in a wider buffer; queries and keys are written over their own inputs
        wide = torch.full((t, (hq + 2 * hk) * d + 64), 7.0, dtype=dt, device="cuda")
        inner = wide[:, :(hq + 2 * hk) * d]
        inner.copy_(rows.view(t, -1))
        heads = inner.unflatten(1, (hq + 2 * hk, d))
        q, k = heads[:, :hq], heads[:, hq:hq + hk]
        plan.run(inner, dev(wq), dev(wk), positions, q, k=k)
        check(q.cpu(), q_ref, bq, "q")
        check(k.cpu(), k_ref, bk, "k")
        assert torch.equal(heads[:, hq + hk:], rows[:, hq + hk:]) and bool((wide[:, (hq + 2 * hk) * d:] == 7).all())
        return
    q = torch.full((t, hq, d), float("nan"), dtype=dt, device="cuda")
    if form == "packed":
        k = torch.full((t, hk, d), float("nan"), dtype=dt, device="cuda")
        plan.run(rows, dev(wq), dev(wk), positions, q, k=k)
        check(q.cpu(), q_ref, bq, "q")
        check(k.cpu(), k_ref, bk, "k")
        return
    for page, order in ((16, "tokens"), (5, "heads")):
        pages = -(-t // page) + 2
        shape = (pages, page, hk, d) if order == "tokens" else (pages, hk, page, d)
        kc, vc = (torch.full(shape, 9.0, dtype=dt, device="cuda") for _ in range(2))
        view = (lambda x: x) if order == "tokens" else (lambda x: x.transpose(1, 2))
        slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(1))[:t]
        slots[::3] = torch.where(torch.arange(len(slots[::3])) % 2 == 1, pages * page + 3, slots[::3])  # outside: not written
        if t > 4:
            slots[4] = -1
        plan.run(rows.view(t, -1), dev(wq), dev(wk), positions, q, k_cache=view(kc), v_cache=view(vc), slots=slots.cuda())
        check(q.cpu(), q_ref, bq, "q")
        flat_k, flat_v = (view(x).reshape(pages * page, hk, d).cpu() for x in (kc, vc))
        inside = (slots >= 0) & (slots < pages * page)
        check(flat_k[slots[inside]], k_ref[inside], bk[inside], "k in the cache")
        assert torch.equal(flat_v[slots[inside]], qkv[inside][:, hq + hk:])
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[slots[inside]] = False
        assert bool((flat_k[rest] == 9).all()) and bool((flat_v[rest] == 9).all())


def test_far_positions_lose_nothing(agmm):
    """Angles at 2^31 and beyond (int64 positions), where a float32 angle would be noise."""
    case = (4, 2, 1, 64, 64, None, False, False, torch.float16, True)
    qkv, wq, wk, _ = _inputs(case, 8)
    pos = torch.tensor([[2 ** 31 - 1, 2 ** 31 + 12345, 2 ** 33 + 7, 10 ** 9]])
    q_ref, k_ref, _, bq, bk = _ref(agmm, case, qkv, wq, wk, pos)
    q, k = torch.empty((4, 2, 64), dtype=torch.float16, device="cuda"), torch.empty((4, 1, 64), dtype=torch.float16, device="cuda")
    _plan(agmm, case).run(qkv.cuda(), wq.cuda(), wk.cuda(), pos.cuda(), q, k=k)
    # both sides round pos * inv_freq in float64: 2^33 * 2^-52 radians
    check(q.cpu(), q_ref, bq + 1e-5, "q")
    check(k.cpu(), k_ref, bk + 1e-5, "k")


def test_extreme_values(agmm):
    """A head of zeros stays zero, a tiny one is lifted by its norm as the formula says, inf and NaN stay in their own head."""
    case = (4, 4, 1, 128, 128, None, False, False, torch.bfloat16, True)
    qkv, wq, wk, pos = _inputs(case, 5)
    qkv[0, 0] = 0
    qkv[1, 1] = 1e-20
    qkv[2, 2, 5] = float("inf")
    qkv[3, 4, 9] = float("nan")
    q_ref, k_ref, _, bq, bk = _ref(agmm, case, qkv, wq, wk, pos)
    q, k = agmm.qkv_norm_rope(qkv.cuda().view(4, -1), wq.cuda(), wk.cuda(), pos.cuda(), 4, 1, base=1e6)
    q, k = q.cpu(), k.cpu()
    assert bool((q[0, 0] == 0).all())
    clean = torch.ones(4, 4, dtype=torch.bool)
    clean[2, 2] = False
    check(q[clean], q_ref[clean], bq[clean], "q")
    check(k[:3], k_ref[:3], bk[:3], "k")
    assert bool(torch.isnan(q[2, 2]).any()) and bool(torch.isnan(k[3]).any())


def test_on_another_stream_and_empty(agmm):
    case = CASES[2]
    t, hq, hk, d = case[:4]
    qkv, wq, wk, pos = _inputs(case, 6)
    q_ref, k_ref, _, bq, bk = _ref(agmm, case, qkv, wq, wk, pos)
    args = [x.cuda() for x in (qkv.view(t, -1), wq, wk, pos)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q, k = agmm.qkv_norm_rope(*args, hq, hk, sections=case[5], base=1e6, stream=s)
    s.synchronize()
    check(q.cpu(), q_ref, bq, "q")
    check(k.cpu(), k_ref, bk, "k")
    q, k = agmm.qkv_norm_rope(args[0][:0], args[1], args[2], args[3][:, :0].contiguous(), hq, hk, sections=case[5])
    assert q.shape == (0, hq, d) and k.shape == (0, hk, d)


def test_refusals(agmm):
    t, hq, hk, d = 3, 4, 2, 64
    plan = agmm.NormRopePlan(hq, hk, d)
    dt = torch.bfloat16
    new = lambda *s, dtype=dt: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    qkv, w, pos, q, k = new(t, (hq + 2 * hk) * d), new(d), new(t, dtype=torch.int32), new(t, hq, d), new(t, hk, d)
    cache, slots = new(2, 16, hk, d), new(t, dtype=torch.int64)
    plan.run(qkv, w, w, pos, q, k=k)
    for bad in (
        lambda: plan.run(new(t, 100), w, w, pos, q, k=k),
        lambda: plan.run(qkv.half(), w, w, pos, q, k=k),
        lambda: plan.run(qkv.cpu(), w, w, pos, q, k=k),
        lambda: plan.run(qkv, w, None, pos, q, k=k),
        lambda: plan.run(qkv, w[:32], w, pos, q, k=k),
        lambda: plan.run(qkv, w.float(), w, pos, q, k=k),
        lambda: plan.run(qkv, w, w, pos[:2], q, k=k),
        lambda: plan.run(qkv, w, w, pos.float(), q, k=k),
        lambda: plan.run(qkv, w, w, pos, q[:2], k=k),
        lambda: plan.run(qkv, w, w, pos, q, k=k[:, :1]),
        lambda: plan.run(qkv, w, w, pos, q, k_cache=cache, v_cache=cache),
        lambda: plan.run(qkv, w, w, pos, q, k_cache=cache, v_cache=cache[:1], slots=slots),
        lambda: plan.run(qkv, w, w, pos, q, k_cache=cache, v_cache=cache, slots=slots.int()),
        lambda: agmm.NormRopePlan(hq, hk, d, sections=(3, 4)),
        lambda: agmm.NormRopePlan(hq, hk, d, inv_freq=[1.0]),
    ):
        with pytest.raises(ValueError):
            bad()
    status = lambda f: pytest.raises(agmm.AgmmError, f).value.status  # noqa: E731
    assert status(lambda: plan.run(qkv, w, w, pos, q)) == agmm.AGMM_ERR_INVALID_ARG  # the keys go nowhere
    odd = new(t * hq * d + 8)[1:1 + t * hq * d].view(t, hq, d)
    assert status(lambda: plan.run(qkv, w, w, pos, odd, k=k)) == agmm.AGMM_ERR_ALIGNMENT
    assert status(lambda: agmm.NormRopePlan(hq, hk, 80)) == agmm.AGMM_ERR_UNSUPPORTED
    assert status(lambda: agmm.NormRopePlan(hq, hk, d, rotary_dim=24)) == agmm.AGMM_ERR_INVALID_ARG
    assert status(lambda: agmm.NormRopePlan(0, hk, d)) == agmm.AGMM_ERR_INVALID_ARG
    assert status(lambda: agmm.NormRopePlan(hq, hk, d, eps=-1.0)) == agmm.AGMM_ERR_INVALID_ARG
    assert status(lambda: agmm.NormRopePlan(hq, hk, d, sections=(8, 8, 8, 4, 4))) == agmm.AGMM_ERR_INVALID_ARG
