"""The activations value by value against 64 bits (GPU only): small negative results, which a bound
relative to z does not see, through each kernel of the linear layer."""
import math

import pytest
import torch

import ops_reference as ref
import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


def exact(z, act):
    """act(z) in 64 bits, of full relative precision for negative z too."""
    z = z.double()
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    u = {"silu": z, "gelu_tanh": 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)}[act]
    return z * torch.exp(u.clamp_max(0)) / (1 + torch.exp(-u.abs()))


def argument(z, act):
    """|log2| of the exponential that makes act(z) small."""
    z = z.double()
    u = {"silu": z, "gelu_tanh": 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3),
         "gelu": z * z / 2}[act]
    return u.abs() / math.log(2)


def through(z, act, out, pre_rows=1):
    """act of z by a product with 1, the values along the rows or the columns of the output."""
    one = torch.ones(1, 1, dtype=z.dtype, device="cuda")
    if pre_rows == 1:
        return tp.linear(one, z[:, None], act=act, out_dtype=out)[0]
    return tp.linear(z[:, None], one, act=act, out_dtype=out)[:, 0]


# Relative error. gelu: of the fit of its tail, 3.5e-4 for 32-bit results and 1.2e-3 for 16-bit ones.
# Elsewhere a few roundings (2^-20) and the exponent's, which is 2^-24 of it before the product that
# makes it adds a few more. A factor below 2^-126 is 0, and below it precision ends.
def bound(z, act, out):
    y = exact(z, act).abs()
    rel = (3.6e-4 if out is F32 else 1.25e-3) if act == "gelu" else 2.0 ** -20
    rel = rel + argument(z, act) * 2.0 ** -22
    return rel * y + ref.U[out] * y + ref.TINY[out] + (1 + z.double().abs()) * 2.0 ** -126


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
def test_small_results_keep_their_size(act, dtype, out):
    z = torch.cat([torch.arange(0, 16.0, 1 / 128), torch.arange(16.0, 100.0, 0.5)]).cuda().neg().to(dtype)
    for rows in (1, len(z)):
        ok, why = ref.within(through(z, act, out, rows), exact(z, act), bound(z, act, out))
        assert ok, why


@pytest.mark.parametrize("path", ["tile", "split"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_each_kernel_alike(path, act, tune):
    z = torch.arange(-14.0, 14.0, 1 / 64, device="cuda").to(BF16)
    few = through(z, act, F32)
    tune.setenv("TPGEMM_LINEAR_PATH", path)
    assert torch.equal(through(z, act, F32), few)
    assert torch.equal(through(z, act, F32, len(z)), few)
    tune.delenv("TPGEMM_LINEAR_PATH")


def test_gelu_is_within_its_absolute_bound():
    # 5.5e-8 of the tail, 5e-8 of its product with |z|, and the rounding of a 32-bit output.
    z = torch.linspace(-16, 16, 20001, device="cuda").to(BF16)
    y = through(z, "gelu", F32)
    ok, why = ref.within(y, exact(z, "gelu"), 6e-8 + 2.0 ** -23 * z.double().abs())
    assert ok, why


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_small_derivatives(act):
    # dZ = act'(Z) through dbias of one row: terms cancel near the derivative's zero, so the bound
    # is of the largest term, and relative past it.
    z = torch.arange(-13.0, 13.0, 1 / 32, device="cuda").to(BF16)
    n = len(z)
    one = torch.ones(1, n, dtype=BF16, device="cuda")
    A, W = torch.zeros(1, 8, dtype=BF16, device="cuda"), torch.zeros(n, 8, dtype=BF16, device="cuda")
    got = tp.linear_backward(one, A, W, z[None], act=act, grad_dtype=F32, need=(False, False, True))[2]
    d = z.double()
    if act == "gelu":
        phi = torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
        terms = [0.5 * torch.erfc(-d / math.sqrt(2)), d * phi]
    else:
        c, q = math.sqrt(2 / math.pi), 0.044715
        u, du = (d, 1.0) if act == "silu" else (2 * c * (d + q * d ** 3), 2 * c * (1 + 3 * q * d * d))
        s = torch.exp(u.clamp_max(0)) / (1 + torch.exp(-u.abs()))
        terms = [s, d * s * torch.exp((-u).clamp_max(0)) / (1 + torch.exp(-u.abs())) * du]
    size = terms[0].abs() + terms[1].abs()
    rel = (1.25e-3 if act == "gelu" else 2.0 ** -19) + argument(z, act) * 2.0 ** -21
    floor = (1 + d.abs() * (1 + 6 * d * d * (act == "gelu_tanh"))) * 2.0 ** -126
    ok, why = ref.within(got, terms[0] + terms[1], rel * size + floor)
    assert ok, why


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("rows", [1, 20, 300])
def test_infinities_follow_the_formulas(act, rows):
    # act(+inf) is inf; act(-inf) is -inf (none), 0 (relu) or, of -inf times 0, a NaN. The largest
    # finite values are not infinite.
    inf, top = float("inf"), torch.finfo(BF16).max
    low = {"none": -inf, "relu": 0.0}.get(act, float("nan"))
    want = torch.tensor([inf, low, top, {"none": -top}.get(act, 0.0), float("nan")], device="cuda")
    z = torch.tensor([inf, -inf, top, -top, float("nan")], device="cuda").to(BF16)
    z = z.repeat(rows, 1)
    one, zero = torch.ones(5, 1, dtype=BF16, device="cuda"), torch.zeros(rows, 1, dtype=BF16, device="cuda")
    for out in (BF16, F32):
        pre = torch.empty(rows, 5, dtype=out, device="cuda")
        # the values come in by the bias of a product that is 0, a row at a time alike
        y = tp.linear(zero, one, z[0].to(out), act=act, out_dtype=out, pre=pre)
        assert torch.equal(torch.nan_to_num(pre.float(), 7.0), torch.nan_to_num(z.float(), 7.0))
        assert torch.equal(torch.isnan(y), torch.isnan(want).expand(rows, 5))
        assert torch.equal(torch.nan_to_num(y.float(), 7.0), torch.nan_to_num(want.to(out).float(), 7.0).expand(rows, 5))


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_derivatives_of_large_values_are_zero_and_one(act):
    z = torch.tensor([[100.0, 1e4, 1e10, 1e20, 3e38]], device="cuda").to(BF16)
    dY, W = torch.ones(1, 5, dtype=BF16, device="cuda"), torch.eye(5, dtype=BF16, device="cuda")
    A = torch.ones(1, 5, dtype=BF16, device="cuda")
    for pre, want in ((z, 1.0), (-z, 0.0)):
        for g in tp.linear_backward(dY, A, W, pre, act=act, grad_dtype=F32):
            assert (g == want).all()
