"""Row scales of the norm where h gamma leaves 32 bits and h rstd gamma does not (GPU only)."""
import pytest
import torch

import ops_reference as ref
import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


# h and gamma of either size: their product is infinite, or below the normal numbers.
@pytest.mark.parametrize("h,gamma", [(1e15, 1e28), (1e-17, 1e-25)])
@pytest.mark.parametrize("cols", [40, 1001, 1024, 8192, 16384, 20000, 20001])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.float8_e5m2])
def test_row_scales_of_products_out_of_range(h, gamma, cols, dtype, kind):
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (torch.randn(5, cols, generator=g, device="cuda") * h).to(dtype)
    x[2] *= 1e-3  # a row of another size
    w = ((1 + 0.2 * torch.randn(cols, generator=g, device="cuda")) * gamma).to(dtype)
    n = tp.rmsnorm(x, w, eps=0.0, quant="row", out_dtype=kind)
    y, _, _ = ref.rmsnorm(x, w, None, 0.0)
    top = ref.FP8[kind][0]
    # sum of squares, square root, division and two products in 32 bits
    e = ref.acc(8 * cols) / 2 + 2.0 ** -20
    want = (y.abs().amax(1) / top).clamp_min(2.0 ** -126)
    ok, why = ref.within(n.scale, want, 2 * e * want)
    assert ok, "scale: " + why
    v = (y / n.scale.double()[:, None]).clamp(-top, top)
    q = n.y.double()
    half = torch.maximum(ref.quantum(v, kind), ref.quantum(q, kind)) / 2
    ok, why = ref.within(q, v, half * (1 + 2.0 ** -10) + 4 * e * v.abs())
    assert ok, "codes: " + why
