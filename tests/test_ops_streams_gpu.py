"""Calls on a given stream while the current one is busy (GPU only): an output is never memory that
work on the current stream still reads, and a dropped one does not come back while its stream writes."""
import pytest
import torch

import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

N = 1024
LONG = 100_000_000  # clocks of a pause: about 50 ms


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


def calls():
    """Name, and a call whose largest outputs are [N, N] of 16 bits (32 of the multiplies)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.randn(N, N, generator=g, device="cuda").half() for _ in range(2))
    w, rstd = torch.ones(N, device="cuda").half(), torch.ones(N, device="cuda")
    a8, b8 = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    sf = torch.full((N, N // 32), 127, dtype=torch.uint8, device="cuda")
    return {"gemm": lambda s: tp.gemm(a, b, stream=s),
            "gemm_mx": lambda s: tp.gemm_mx(a8, b8, sf, sf, stream=s),
            "linear": lambda s: tp.linear(a, b, stream=s),
            "linear_backward": lambda s: tp.linear_backward(a, a, b, stream=s)[1],
            "rmsnorm": lambda s: tp.rmsnorm(a, w, b, need_rstd=True, stream=s).h,
            "rmsnorm_backward": lambda s: tp.rmsnorm_backward(a, b, rstd, w, stream=s)[0]}


NAMES = ["gemm", "gemm_mx", "linear", "linear_backward", "rmsnorm", "rmsnorm_backward"]


@pytest.mark.parametrize("kind", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_taken_from_the_current_stream(name, kind):
    call = calls()[name]
    s = torch.cuda.Stream()
    given = s if kind == "stream" else s.cuda_stream
    want = call(None).clone()
    call(given)  # modules loaded, memory of both streams at hand
    torch.cuda.synchronize()
    blocks = [torch.full((N, N), float(i), dtype=want.dtype, device="cuda") for i in range(8)]
    copies = [torch.empty_like(b) for b in blocks]
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    for c, b in zip(copies, blocks):
        c.copy_(b)  # still to run when the blocks are given back
    del b, blocks
    got = [call(given) for _ in range(4)]
    torch.cuda.synchronize()
    for i, c in enumerate(copies):
        assert (c == i).all()
    assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("name", NAMES)
def test_dropped_outputs_do_not_come_back_to_the_current_stream(name):
    call = calls()[name]
    s = torch.cuda.Stream()
    dtype = call(s).dtype
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(LONG)
    for _ in range(4):
        call(s)  # its result is dropped before it has run
    mine = [torch.full((N, N), float(i), dtype=dtype, device="cuda") for i in range(16)]
    torch.cuda.synchronize()
    for i, m in enumerate(mine):
        assert (m == i).all()


def test_the_default_stream_by_its_handles():
    call = calls()["linear"]
    want = call(None).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (0, 1):
        with torch.cuda.stream(s):
            got = call(handle)
            assert torch.cuda.current_stream() == s
        torch.cuda.synchronize()
        assert torch.equal(got, want)
