"""The functions' own buffers belong to the stream they are given, in whatever form it comes.

Memory that a workspace may get held other bytes before, and the current stream is busy
for about 100 ms: a workspace that was zeroed there would not be zero when the kernel
reads it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


class Handle:
    """Another library's stream object."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


FORMS = {
    "stream": lambda s: s,
    "handle": lambda s: s.cuda_stream,
    "object": Handle,
    "external": lambda s: torch.cuda.ExternalStream(s.cuda_stream),
}


@pytest.fixture(scope="module")
def agmm():
    import all_gather_gemm_agmm_gb300 as m
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    m.load_library()
    return m


def _calls(agmm):
    g = torch.Generator(device="cuda").manual_seed(2)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rows, positions = new(300, 16 * 64), torch.arange(300, device="cuda")[None]
    q, k, v, starts = new(1200, 16, 64), new(1200, 4, 64), new(1200, 4, 64), ints(list(range(0, 1201, 40)))
    drafts, kc, vc = new(6, 16, 64), new(60, 64, 4, 64), new(60, 64, 4, 64)
    table, ctx, nodes = torch.arange(60, dtype=torch.int32, device="cuda").view(2, 30), ints([1800, 77]), ints([0, 3, 6])
    one = ints([0, 1000])
    return {
        "rope": lambda **kw: agmm.qkv_norm_rope(rows, None, None, positions, 8, 4, **kw),
        "prompt": lambda **kw: (agmm.prompt_attention(q, k, v, starts, **kw),),  # drawn
        "cut prompt": lambda **kw: (agmm.prompt_attention(q[:1000], k[:1000], v[:1000], one, **kw),),
        "tree": lambda **kw: (agmm.tree_attention(drafts, kc, vc, table, ctx, nodes, max_nodes=3, **kw),),
    }


def _same(got, want):
    return len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def _dirty():
    """Free blocks of the current stream that hold large numbers, for workspaces and outputs to be made in."""
    for mb in (1, 2, 4, 8, 16, 32, 48, 64):
        torch.full((mb << 20,), 0x3f, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("name", ["rope", "prompt", "cut prompt", "tree"])
def test_buffers_belong_to_the_given_stream(agmm, name, form):
    call = _calls(agmm)[name]
    want = call()
    _dirty()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    busy = torch.cuda.Event()
    busy.record()
    got = call(stream=FORMS[form](s))
    s.synchronize()
    assert not busy.query(), "the call waited for the current stream"
    torch.cuda.synchronize()
    assert _same(got, want)


def test_what_a_call_frees_stays_with_its_stream(agmm):
    """The workspace of a call on a handle is not handed to the current stream while the kernel may use it."""
    call = _calls(agmm)["prompt"]
    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    outs = []
    for _ in range(3):
        outs.append(call(stream=s.cuda_stream))  # waits behind the sleep
        _dirty()                                 # runs at once, in whatever memory is free
    torch.cuda.synchronize()
    assert all(_same(o, want) for o in outs)


@pytest.mark.parametrize("name", ["rope", "prompt", "tree"])
def test_the_default_stream_by_its_handle(agmm, name):
    call = _calls(agmm)[name]
    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):  # current; the call is for another one
        got = call(stream=0)
    torch.cuda.synchronize()
    assert _same(got, want)


@pytest.mark.parametrize("handle", [1, 2], ids=["legacy", "per-thread"])
@pytest.mark.parametrize("name", ["rope", "prompt", "tree"])
def test_the_special_handles(agmm, name, handle):
    """cudaStreamLegacy and cudaStreamPerThread, while the current stream is another one and busy."""
    call = _calls(agmm)[name]
    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        _dirty()
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)
        got = call(stream=handle)
    torch.cuda.synchronize()
    assert _same(got, want)
