"""32-bit gradients of the gated linear layer against 64 bits, by bounds that leave no room for a dZ of
16 bits or an activation made for 16-bit results (GPU only): every activation, more tokens than one
sum takes, infinities, and sums of 32-bit outputs that are longer than their pieces."""
import math

import pytest
import torch

import more_ops_reference as more
import ops_reference as ref
import test_gated_linear_gpu as gl
import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E32 = more.E32


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


def dz_of(dY, pre, act):
    """dZ in 64 bits, and what the 32-bit one is off by. Activations are as of 32-bit outputs (silu and
    gelu_tanh within 2^-20 of themselves and 2^-22 |log2 f| more; gelu within 6e-8, 5e-6 of itself down
    to -3 and 4e-4 below); their derivatives, whose terms cancel, are absolute: 2^-18, and of gelu, the
    sum of a tail within 5.5e-8 and of a product of at most 0.25 within 2^-21 of itself, 2^-21."""
    dy = dY.double()
    g, u = pre.double().chunk(2, 1)
    f, df = ref.act(g, act), ref.act_grad(g, act)
    if act == "gelu_tanh":  # (1 + tanh v as it stands loses its digits where it is small, in 64 bits too)
        f = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    zero = torch.zeros_like(g)
    if act == "gelu":
        ef = torch.minimum(torch.full_like(g, 6e-8), torch.where(g >= -3, 5e-6, 4e-4) * f.abs())
        ed = zero + 2.0 ** -21
    elif act in ("silu", "gelu_tanh"):
        factor = torch.where(g == 0, 0.5, f / torch.where(g == 0, 1.0, g)).clamp_min(2.0 ** -126)
        ef = (2.0 ** -20 + 2.0 ** -22 * factor.log2().abs()) * f.abs()
        ed = zero + 2.0 ** -18
    else:
        ef = ed = zero
    dz = torch.cat([dy * u * df, dy * f], 1)
    err = torch.cat([(dy * u).abs() * ed, dy.abs() * ef], 1) + 4 * E32 * dz.abs()
    return dz, err


def check(dY, A, W, pre, act):
    _, dW, db = tp.gated_linear_backward(dY, A, W, pre, act=act, grad_dtype=F32)
    dz, err = dz_of(dY, pre, act)
    # two 16-bit values of dz: 2^-17 of it, and half of f16's last step, 2^-25, of the rest, which is
    # kept 2^11 times as large
    split = err + 2.0 ** -17 * dz.abs() + (2.0 ** -36 if dY.dtype is F16 else 0.0)
    a, M = A.double(), A.shape[0]
    want, terms = dz.t() @ a, dz.abs().t() @ a.abs()
    ok, why = ref.within(dW, want, split.t() @ a.abs() + 2 * ref.acc(M) * terms + 4 * E32 * want.abs() + 1e-44)
    assert ok, "dW: " + why
    ok, why = ref.within(db, dz.sum(0), err.sum(0) + ref.acc(8 * M) * dz.abs().sum(0) + 1e-44)
    assert ok, "dbias: " + why


def args(M, N, K, dtype, seed, pad=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (gl.view(g, M, N, dtype, pad, std=std), gl.view(g, M, K, dtype, pad), gl.view(g, 2 * N, K, dtype, pad),
            gl.view(g, M, 2 * N, dtype, pad, std=1.5))


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K,pad", [(3, 72, 256, 0), (100, 72, 264, 0), (100, 33, 65, 0), (700, 264, 136, 3)])
def test_weight_and_bias_gradients(M, N, K, pad, dtype, act):
    check(*args(M, N, K, dtype, M, pad), act)


@pytest.mark.parametrize("dtype,std", [(F16, 1e-5), (BF16, 1e-25), (BF16, 1e25)])
def test_small_and_large(dtype, std):
    check(*args(300, 72, 136, dtype, 7, std=std), "silu")


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("M", [4096, 4097, 8191, 10000])
@pytest.mark.parametrize("N,K,pad", [(40, 72, 0), (33, 65, 1), (264, 136, 0)])
def test_more_tokens_than_a_sum_takes(M, N, K, pad, act):
    for dtype in (F16, BF16):
        check(*args(M, N, K, dtype, M, pad), act)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M", [64, 600])
def test_negative_gates(M, dtype, act):
    # One gate to a column, terms of one sign: what an activation is off by, relative to itself, all of
    # the column's terms are off by alike.
    gates = torch.linspace(-3, -1, 64, device="cuda").to(dtype)
    g = torch.Generator(device="cuda").manual_seed(M)
    pre = torch.cat([gates.expand(M, 64), 0.5 + torch.rand(M, 64, generator=g, device="cuda").to(dtype)], 1)
    dY, A = ((0.5 + torch.rand(M, n, generator=g, device="cuda")).to(dtype) for n in (64, 72))
    check(dY, A, gl.view(g, 128, 72, dtype), pre, act)


@pytest.mark.parametrize("path", ["tile", "split"])
@pytest.mark.parametrize("M,N,K", [(100, 40, 264), (300, 40, 265), (5000, 72, 136)])
@pytest.mark.parametrize("whole", [True, False])
def test_infinities_of_the_input(M, N, K, whole, path, tune):
    # An infinite A[m, k] makes column k of dW infinite with dZ[m]'s signs, whether dZ is a 16-bit value
    # (whole numbers) or not, and a second one of the other sign a NaN where those signs agree.
    tune.setenv("TPGEMM_LINEAR_PATH", path)
    for dtype in (F16, BF16):
        dY, A, W, pre = args(M, N, K, dtype, 3)
        if whole:
            dY, pre = dY.sign() + (dY == 0), (pre * 4).round() + (pre.abs() <= 0.125)
        A[7, 5], A[M - 1, 5], A[M - 2, 9] = float("inf"), float("-inf"), float("-inf")
        _, dW, _ = tp.gated_linear_backward(dY, A, W, pre, act="none", grad_dtype=F32)
        dz, _ = dz_of(dY, pre, "none")
        assert (dz[[7, M - 1, M - 2]] != 0).all()
        assert torch.equal(dW[:, 9].double(), dz[M - 2].sign() * float("-inf"))
        meet = dz[7].sign() * float("inf") + dz[M - 1].sign() * float("-inf")
        assert torch.equal(torch.isnan(dW[:, 5]), torch.isnan(meet))
        assert torch.equal(dW[:, 5].double()[~torch.isnan(meet)], meet[~torch.isnan(meet)])
        rest = [k for k in range(K) if k not in (5, 9)]
        clean = A.clone()
        clean[:, [5, 9]] = 0
        _, want, _ = tp.gated_linear_backward(dY, clean, W, pre, act="none", grad_dtype=F32)
        assert torch.equal(dW[:, rest], want[:, rest])


@pytest.mark.parametrize("M,K,share", [(1100, 5000, 2560), (40, 32768, 4096), (40, 65536, 8192)])
def test_long_sums_of_32_bit_outputs(M, K, share):
    # Sums come in at most eight pieces. A term of a piece costs its sum up to 1.2e-9 of its size, and
    # an output is a product of two sums.
    g = torch.Generator(device="cuda").manual_seed(K)
    A, W = gl.view(g, M, K, BF16), gl.view(g, 200, K, BF16, std=K ** -0.5)
    y = tp.gated_linear(A, W, act="none", out_dtype=F32)
    z = A.double() @ W.double().t()
    want = z[:, :100] * z[:, 100:]
    # (two sums, and a rounding of each and of the product)
    assert float((y.double() - want).norm() / want.norm()) <= 2 * 1.2e-9 * share + 3 * E32
