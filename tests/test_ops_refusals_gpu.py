"""Refusals of the operators around the multiply in Python that need tensors on the GPU."""
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
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


def half(*shape):
    return torch.ones(shape, device="cuda").half()


@pytest.mark.parametrize("shape", [(), (16,), (1, 8, 16)])
def test_weights_that_are_no_matrix(shape):
    for call in (lambda: tp.linear(half(4, 16), half(*shape)),
                 lambda: tp.linear_backward(half(4, 8), half(4, 16), half(*shape))):
        with pytest.raises(ValueError, match="W must be 2-D"):
            call()


def test_a_workspace_with_gaps():
    # Its elements' bytes from its start on would be used, which are not all its own.
    A, W, dY, w = half(40, 41), half(24, 41), half(40, 24), half(41)
    whole = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    ok = tp.linear(A, W, workspace=whole)
    assert torch.equal(ok, tp.linear(A, W))
    whole.zero_()
    for call in (lambda ws: tp.linear(A, W, workspace=ws), lambda ws: tp.linear_backward(dY, A, W, workspace=ws),
                 lambda ws: tp.rmsnorm_backward(A, A, torch.ones(40, device="cuda"), w, workspace=ws)):
        with pytest.raises(ValueError, match="contiguous"):
            call(whole[::2])
    torch.cuda.synchronize()
    assert (whole == 0).all()
