"""The bounded waits of the linear layer's tcgen05 kernels (GPU only): their bound begins when the
previous grid has ended, and a bound that is too short for the work ends the kernel with a status."""
import pytest
import torch

import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


def ones(g, *shape):
    """Values of -1, 0 and 1: sums of up to 256 of their products are exact in bfloat16."""
    return torch.randint(-1, 2, shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("path,M,N", [("tile", 512, 512), ("split", 40, 512), ("split", 512, 40)])
def test_no_bound_runs_while_the_previous_grid_does(path, M, N, tune):
    # A multiply on two of the GPU's SMs, milliseconds long with waits of microseconds, and behind
    # it a small product that may start on the others at once, under a bound of 3 ms.
    g = torch.Generator(device="cuda").manual_seed(M)
    A, W = ones(g, M, 256), ones(g, N, 256)
    want = (A.float() @ W.float().t()).bfloat16()
    big = torch.zeros(4096, 4096, device="cuda").bfloat16()
    out = torch.empty(4096, 4096, device="cuda")
    tune.setenv("TPGEMM_LINEAR_PATH", path)
    tp.linear(A, W)
    torch.cuda.synchronize()
    tune.setenv("TPGEMM_TC_MAX_CLUSTERS", "1")
    tune.setenv("TPGEMM_TC_SK", "0")
    tune.setenv("TPGEMM_WAIT_TIMEOUT_MS", "3")
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    tp.gemm(big, big, transB=True, out=out)
    got = tp.linear(A, W)
    end.record()
    torch.cuda.synchronize()
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK
    assert begin.elapsed_time(end) > 4.0  # (else nothing was shown)
    assert torch.equal(got, want)
