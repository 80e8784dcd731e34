"""Every kernel variant of the feed-forward products, at small sizes: wide and narrow row tiles,
whole, cut and shared by pairs, and swapped tiles whose k is shared by 1 to 8 CTAs.  The rules choose among them by
size; here the overrides do."""
import pytest
import torch

from feedforward_ref import check, gated, gated_grad, linear, linear_grad

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


ROWS = [dict(AGMM_PATH="0", AGMM_BN=bn, AGMM_STREAMK=cut) for bn in ("128", "256") for cut in ("0", "1")]
ROWS += [dict(AGMM_PATH="0", AGMM_BN="128", AGMM_SPLITK=str(s)) for s in (2, 3, 4)]
ROWS += [dict(AGMM_PATH="0", AGMM_BN=bn, AGMM_MERGE=m) for bn in ("128", "256") for m in ("0", "1")]
SWAP = [dict(AGMM_PATH="1", AGMM_SPLITK=str(s)) for s in (1, 2, 3, 4, 5, 6, 7, 8)]


def name(env):
    return "-".join(k[5:].lower() + v for k, v in env.items())


# shards, rows, k, n: one row to several tiles, sizes that end inside tiles and k blocks
SIZES = [(1, 1, 1000, 264), (3, 13, 584, 136), (8, 7, 520, 264), (2, 200, 1032, 648)]


@pytest.mark.parametrize("env", ROWS + SWAP, ids=name)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("transpose", [False, True])
def test_paths(agmm, monkeypatch, env, size, transpose):
    shards, rows, k, n = size
    if env["AGMM_PATH"] == "1" and shards * (-(-rows // 8) * 8) > 64:
        pytest.skip("more tokens than a swapped tile has")
    for e, v in env.items():
        monkeypatch.setenv(e, v)
    dtype = torch.float16 if transpose else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(8)
    new = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
    t = shards * rows
    shape = (n, k) if transpose else (k, n)
    xs, wg, wu = [new(rows, k) for _ in range(shards)], new(*shape, std=k ** -0.5), new(*shape, std=k ** -0.5)
    x, d, r, b, z = torch.cat(xs), new(t, n), new(t, n), new(n), new(t, n)
    nan = lambda *s: torch.full(s, float("nan"), dtype=dtype, device="cuda")  # noqa: E731

    plan = agmm.GatedPlan(k, n, activation="silu", rhs_transpose=transpose, f16=transpose)
    ws = plan.new_workspace()
    got = dict(out=nan(t, n), gate=nan(t, n), up=nan(t, n))
    plan.run(xs, wg, wu, got["out"], ws, gate=got["gate"], up=got["up"])
    want = gated(x, wg, wu, "silu", transpose, dtype)
    for key, y in got.items():
        check(y, *want[key], f"gated {key}")
    got = dict(d_gate=nan(t, n), d_up=nan(t, n), dx=nan(t, k), dw_gate=nan(*shape), dw_up=nan(*shape))
    plan.backward(d, xs, wg, wu, z, r, got["d_gate"], got["d_up"], ws, dx=got["dx"], dw_gate=got["dw_gate"], dw_up=got["dw_up"])
    want = gated_grad(d, x, wg, wu, z, r, "silu", transpose, dtype, dtype)
    for key, y in got.items():
        check(y, *want[key], f"gated {key}")

    plan = agmm.LinearPlan(k, n, activation="gelu", rhs_transpose=transpose, f16=transpose)
    got = dict(out=nan(t, n), pre=nan(t, n))
    plan.run(xs, wg, got["out"], ws, bias=b, residual=r, pre=got["pre"])
    want = linear(x, wg, b, r, "gelu", transpose, dtype)
    for key, y in got.items():
        check(y, *want[key], f"linear {key}")
    f32 = torch.empty(shape, device="cuda")
    got = dict(dx=nan(t, k), dw=f32, d_bias=torch.empty(n, device="cuda"))
    plan.backward(d, xs, wg, ws, pre=z, d_pre=nan(t, n), **got)
    want = linear_grad(d, x, wg, z, "gelu", transpose, dtype, torch.float32)
    for key, y in got.items():
        check(y, *want[key], f"linear {key}")
    plan.query_status(ws)


@pytest.mark.parametrize("env", [e for e in ROWS if e.get("AGMM_STREAMK") == "1"], ids=name)
def test_cut_tiles_behind_whole_ones(agmm, monkeypatch, env):
    """More tiles than clusters, the ragged last wave cut: parts of both slots, and whole tiles behind them."""
    for e, v in env.items():
        monkeypatch.setenv(e, v)
    m, k, n = 2560, 456, 2600
    g = torch.Generator(device="cuda").manual_seed(9)
    new = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    x, w, r = new(m, k), new(n, k, std=k ** -0.5), new(m, n)
    plan = agmm.LinearPlan(k, n, rhs_transpose=True)
    ws = plan.new_workspace()
    first = torch.empty_like(r)
    plan.run(x, w, first, ws, residual=r)
    check(first, *linear(x, w, None, r, None, True, torch.bfloat16)["out"], "out")
    for _ in range(10):
        again = torch.full_like(r, float("nan"))
        plan.run(x, w, again, ws, residual=r)
        assert torch.equal(first, again)


@pytest.mark.parametrize("sizes", [(300, 264, 4104), (2000, 4104, 72), (1500, 1032, 1544), (900, 72, 2056)], ids=str)
@pytest.mark.parametrize("bn", ["128", "256"])
def test_both_gradients_in_one_launch(agmm, monkeypatch, sizes, bn):
    """Either product the longer one, few and many tiles of each, as two launches give them bit by bit
    (none of them is cut)."""
    t, k, n = sizes
    g = torch.Generator(device="cuda").manual_seed(10)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, d = [new(t // 2, k) for _ in range(2)], new(k, n), new(t, n)
    monkeypatch.setenv("AGMM_BN", bn)
    monkeypatch.setenv("AGMM_STREAMK", "0")
    monkeypatch.setenv("AGMM_SPLITK", "1")
    got = []
    for merge in ("0", "1"):
        monkeypatch.setenv("AGMM_MERGE", merge)
        plan = agmm.LinearPlan(k, n)
        ws = plan.new_workspace()
        dx, dw = torch.full((t, k), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.full((k, n), float("nan"), device="cuda")
        plan.backward(d, x, w, ws, dx=dx, dw=dw)
        plan.query_status(ws)
        got.append((dx, dw))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    want = linear_grad(d, torch.cat(x), w, None, None, False, torch.bfloat16, torch.float32)
    check(got[1][0], *want["dx"], "dx")
    check(got[1][1], *want["dw"], "dw")
