"""The product's own buffers belong to the stream that all_gather_matmul is given.

The kernels count arrivals in the workspace from zero: one that is zeroed on another
stream, which is busy for about 100 ms here, is not zero when they read it."""
import pytest
import torch

from test_gpu_attention_streams import FORMS, _dirty

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("m,k,n,unfused", [(64, 4096, 1024, False), (512, 1024, 2048, False), (64, 1024, 512, True)], ids=str)
def test_buffers_belong_to_the_given_stream(form, m, k, n, unfused):
    import all_gather_gemm_agmm_gb300 as agmm
    from all_gather_gemm_agmm_gb300 import _build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    g = torch.Generator(device="cuda").manual_seed(m)
    xs = [torch.randn((m, k), generator=g, device="cuda").bfloat16() for _ in range(2)]
    y = torch.randn((n, k), generator=g, device="cuda").bfloat16()
    call = lambda **kw: agmm.all_gather_matmul(xs, y, my_id=1, rhs_transpose=True, unfused=unfused, **kw)  # noqa: E731
    want = call()
    _dirty()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    busy = torch.cuda.Event()
    busy.record()
    got = [call(stream=FORMS[form](s))]
    if not unfused:
        got += agmm.all_gather_matmul(xs, y, my_id=1, rhs_transpose=True, return_gathered=True, stream=FORMS[form](s))
    s.synchronize()
    assert not busy.query(), "the call waited for the current stream"
    torch.cuda.synchronize()
    assert torch.equal(got[0], want)
    if not unfused:
        assert torch.equal(got[1], want) and torch.equal(got[2], torch.cat(xs))
