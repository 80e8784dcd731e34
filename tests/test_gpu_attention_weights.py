"""Many keys of little weight next to one that has most of it, in fp16: their mass is not lost.

Scores are exact: q is the first unit vector, a key's score is its first column.  Bound of
an output sum(p v) / sum(p) with |v| <= 1 and the largest p 1: a weight is held as
an fp16 number 2^7 times as large, so it is off by 2^-11 of itself, or below 2^-21 by 2^-32;
1e-4 covers the float32 arithmetic; the output is rounded once, to 2^-11 of itself or
2^-25."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -11
FAINT = -17.40625  # e^FAINT = 2^-25.11: less than half of fp16's smallest number


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


def _keys(scores, values, d, heads=1):
    """Keys of these scores, and values given by their first columns."""
    k, v = (torch.zeros((len(scores), heads, d), dtype=torch.float16, device="cuda") for _ in range(2))
    k[..., 0] = scores.half()[:, None]
    assert torch.equal(k[:, 0, 0].double(), scores.double().cuda())
    v[..., :values.shape[1]] = values.half()[:, None]
    return k, v


def _want(scores, values):
    """(the output's first columns, their bound)."""
    p = torch.exp(scores.double() - scores.double().max())
    o = p @ values.double() / p.sum()
    size = p @ values.double().abs() / p.sum()
    lost = len(scores) * 2.0 ** -32 / p.sum()
    return o, U * o.abs() + 2.0 ** -25 + (U + 1e-4) * size + (1 + size) * lost


def _near(got, want, bound, what):
    over = float(((got.double().cpu() - want).abs() - bound).max())
    assert over <= 0, f"{what}: {over:.2e} over the bound; {got.tolist()} for {want.tolist()}"


def _sink(n, at):
    scores = torch.full((n,), FAINT, dtype=torch.float64)
    scores[at] = 0.0
    values = torch.zeros((n, 2), dtype=torch.float64)
    values[:, 1] = 1.0
    values[at] = torch.tensor([1.0, 0.0], dtype=torch.float64)
    return scores, values


def _query(rows, heads, d):
    q = torch.zeros((rows, heads, d), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    return q


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 70000, -1])
def test_faint_keys_of_a_long_context(agmm, d, at):
    n, page = 131073, 64
    scores, values = _sink(n, at)
    k, v = _keys(scores, values, d)
    pad = -n % page
    kc, vc = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(-1, page, 1, d) for x in (k, v))
    table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None]
    out = agmm.tree_attention(_query(1, 2, d), kc, vc, table, _ints([n - 1]), _ints([0, 1]), max_nodes=1, scale=1.0)
    want, bound = _want(scores, values)
    for h in range(2):
        _near(out[0, h, :2], want, bound, f"head {h}")


@pytest.mark.parametrize("drawn", [False, True])
def test_faint_keys_of_a_prompt(agmm, drawn):
    """One query behind a prefix, alone (cut along the keys) or among many others (drawn whole)."""
    n, d, heads = 40001, 64, 16
    scores, values = _sink(n, 3)
    k, v = _keys(scores, values, d)
    others = 30 if drawn else 0
    k = torch.cat([k, torch.zeros((others, 1, d), dtype=torch.float16, device="cuda")])
    v = torch.cat([v, torch.zeros((others, 1, d), dtype=torch.float16, device="cuda")])
    starts = _ints(list(range(others + 2)))
    out = agmm.prompt_attention(_query(others + 1, heads, d), k, v, starts, _ints([0] + [n + i for i in range(others + 1)]), scale=1.0)
    want, bound = _want(scores, values)
    for h in range(heads):
        _near(out[0, h, :2], want, bound, f"head {h}")


def test_faint_keys_beside_a_value_that_a_row_does_not_see(agmm):
    """The row is computed again without it, with all of its mass."""
    n, d = 3000, 64
    scores, values = _sink(n, 5)
    k, v = _keys(torch.cat([scores, torch.zeros(1, dtype=torch.float64)]), torch.cat([values, torch.zeros((1, 2), dtype=torch.float64)]), d)
    v[n] = float("nan")
    out = agmm.prompt_attention(_query(2, 4, d), k, v, _ints([0, 2]), _ints([0, n + 1]), scale=1.0)
    want, bound = _want(scores, values)
    for h in range(4):
        _near(out[0, h, :2], want, bound, f"head {h}")
    assert bool(torch.isnan(out[1]).all())


def test_scores_that_grow_by_less_than_the_reference_follows(agmm):
    """The largest weights that are held, times the largest values: neither the weights nor the sums overflow."""
    n, d = 20000, 64
    scores = torch.full((n,), 5.53125, dtype=torch.float64)  # 2^7.98
    scores[:128] = 0.0
    values = torch.full((n, 2), 65504.0, dtype=torch.float64)
    values[::2, 1] = -65504.0
    k, v = _keys(scores, values, d)
    out = agmm.prompt_attention(_query(1, 2, d), k, v, _ints([0, 1]), _ints([0, n]), scale=1.0)
    want, bound = _want(scores, values / 65504.0)
    _near(out[0, 0, :2] / 65504.0, want, bound, "values")
