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


def gives_up(A, W, residual, pre):
    """Whether the product ends with the waits' status, read once, and the context goes on."""
    tp.linear(A, W, None, residual, pre=pre)
    status = tp.tpgemm_last_device_error()
    assert status in (tp.TPGEMM_OK, tp.TPGEMM_ERR_TIMEOUT), tp.tpgemm_last_error_detail()
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK
    return status == tp.TPGEMM_ERR_TIMEOUT


# Sums so long that the epilogue's wait for one runs out on a healthy product, with fills and MMAs
# under way in both CTAs of each pair: all roles stop, what is in flight lands, tensor memory is
# freed, and the next call on the same SMs is right.
@pytest.mark.parametrize("M,N,more", [(256, 256, False), (250, 250, True), (512, 512, True)])
def test_a_tile_product_that_gives_up(M, N, more, tune):
    g = torch.Generator(device="cuda").manual_seed(N)
    K = 1 << (21 if M <= 256 else 20)
    A, W = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") if more else None
    z = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") if more and M == 512 else None
    a, w = ones(g, 1000, 192), ones(g, 1200, 192)
    want = (a.float() @ w.float().t()).bfloat16()
    tune.setenv("TPGEMM_LINEAR_PATH", "tile")
    for i in range(6):
        tune.setenv("TPGEMM_WAIT_TIMEOUT_MS", "1")
        assert gives_up(A, W, r, z)
        tune.delenv("TPGEMM_WAIT_TIMEOUT_MS")
        for _ in range(3):
            assert torch.equal(tp.linear(a, w), want)
    assert not gives_up(A, W, r, z)


@pytest.mark.parametrize("split", [1, 2])
@pytest.mark.parametrize("M,N", [(40, 128), (128, 40)])
def test_a_split_product_that_gives_up(M, N, split, tune):
    g = torch.Generator(device="cuda").manual_seed(split)
    K = 1 << 22
    A, W = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    a, w = ones(g, 100, 192), ones(g, 1200, 192)
    want = (a.float() @ w.float().t()).bfloat16()
    tune.setenv("TPGEMM_LINEAR_PATH", "split")
    tune.setenv("TPGEMM_LINEAR_SPLIT", str(split))
    for i in range(6):
        tune.setenv("TPGEMM_WAIT_TIMEOUT_MS", "1")
        assert gives_up(A, W, None, None)
        tune.delenv("TPGEMM_WAIT_TIMEOUT_MS")
        for _ in range(3):
            assert torch.equal(tp.linear(a, w), want)
    assert not gives_up(A, W, None, None)
