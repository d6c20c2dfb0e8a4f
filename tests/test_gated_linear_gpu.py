"""The gated linear layer and its gradients against 64-bit formulas (GPU only): each kernel by itself,
from one token up, odd and ragged sizes, every type and activation, scales, strides, kept values
before the gate, empty sizes, infinities and NaN, captured calls, and integers exact to the bit."""
import pytest
import torch

import more_ops_reference as more
import ops_reference as ref
import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


def view(g, rows, cols, dtype, pad=0, offset=0, std=1.0):
    ld = cols + pad
    flat = torch.randn(rows * ld + offset, generator=g, device="cuda") * std
    return flat.to(dtype).as_strided((rows, cols), (ld, 1), offset)


def blank(rows, cols, dtype, pad, offset):
    buf = torch.full((rows * (cols + pad) + offset + 64,), 3.0, device="cuda").to(dtype)
    return buf, buf.as_strided((rows, cols), (cols + pad, 1), offset)


def untouched(buf, rows, cols, pad, offset):
    mask = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    mask.as_strided((rows, cols), (cols + pad, 1), offset).fill_(False)
    return bool((buf[mask] == 3).all())


def check(M, N, K, dtype=BF16, act="silu", bias=True, pre=True, out=None, scales=None, pad=0, offset=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f8 = dtype in ref.FP8
    out = out or (BF16 if f8 else dtype)
    scales = f8 if scales is None else scales
    A = view(g, M, K, dtype, pad, offset)
    W = view(g, 2 * N, K, dtype, pad, offset, max(K, 1) ** -0.5 if not f8 else 1.0)
    b = view(g, 1, 2 * N, out)[0] if bias else None
    sa = torch.rand(M, generator=g, device="cuda") + 0.5 if scales else None
    sw = (torch.rand(2 * N, generator=g, device="cuda") + 0.5) * max(K, 1) ** -0.5 if scales else None
    ybuf, y = blank(M, N, out, pad, offset)
    zbuf, z = blank(M, 2 * N, out, pad, offset) if pre else (None, None)
    tp.gated_linear(A, W, b, act=act, scale_a=sa, scale_w=sw, out_dtype=out, out=y, pre=z)
    torch.cuda.synchronize()
    assert untouched(ybuf, M, N, pad, offset) and (not pre or untouched(zbuf, M, 2 * N, pad, offset))
    ry, rz, by, bz = more.gated(A, W, b, act, sa, sw, out)
    if pre:
        ok, why = ref.within(z, rz, bz)
        assert ok, "pre: " + why
    ok, why = ref.within(y, ry, by)
    assert ok, "y: " + why


SIZES = [(1, 1, 1), (1, 8, 64), (1, 512, 4096), (2, 33, 65), (7, 40, 264), (8, 100, 1000), (16, 1024, 512),
         (17, 64, 128), (37, 500, 1001), (64, 48, 2048), (100, 520, 264), (129, 130, 72), (144, 1000, 1032),
         (256, 2048, 512), (300, 36, 4096), (513, 1536, 64), (1000, 7, 256), (1024, 1024, 1024), (2050, 264, 40)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(M, N, K):
    check(M, N, K, seed=M)
    check(M, N, K, F16, bias=False, pre=False, out=F32, seed=N)


@pytest.mark.parametrize("path", ["tile", "split", "few"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (5, 72, 1000), (16, 264, 2048), (40, 136, 512), (200, 96, 264),
                                   (260, 300, 128), (300, 1032, 520)])
def test_each_kernel(path, M, N, K, tune):
    if path == "few" and M > 16:
        pytest.skip("up to 16 tokens")
    tune.setenv("TPGEMM_LINEAR_PATH", path)
    for out in (BF16, F32):
        check(M, N, K, out=out, seed=M)
        check(M, N, K, out=out, bias=False, pre=False, act="gelu", seed=M)
    check(M, N, K, E4M3, seed=M)
    check(M, N, K + 3, F16, seed=M)


@pytest.mark.parametrize("bn", [64, 128, 192, 256])
def test_tile_widths(bn, tune):
    tune.setenv("TPGEMM_LINEAR_PATH", "tile")
    tune.setenv("TPGEMM_LINEAR_BN", str(bn))
    for N in (8, 31, 200, 1000):
        check(600, N, 192, seed=bn)
        check(600, N, 192, out=F32, seed=bn)


@pytest.mark.parametrize("bp", [64, 80, 96, 112, 128])
@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_split_shapes(bp, split, tune):
    tune.setenv("TPGEMM_LINEAR_PATH", "split")
    tune.setenv("TPGEMM_LINEAR_BP", str(bp))
    tune.setenv("TPGEMM_LINEAR_SPLIT", str(split))
    for M, N in ((30, 200), (100, 333), (280, 24)):
        check(M, N, 1024, seed=bp)


@pytest.mark.parametrize("dtype,outs", [(F16, (F16, F32)), (BF16, (BF16, F32)), (E4M3, (F16, BF16, F32)),
                                        (E5M2, (F16, BF16, F32))])
@pytest.mark.parametrize("act", ref.ACTS)
def test_types_and_activations(dtype, outs, act):
    for out in outs:
        for M, N, K in ((3, 72, 256), (40, 136, 272), (520, 320, 128)):
            check(M, N, K, dtype, act, out=out, seed=M)


@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (1, 0), (0, 1), (8, 4), (7, 3)])
@pytest.mark.parametrize("M,N,K", [(3, 72, 256), (60, 100, 264), (300, 264, 96)])
def test_strides_and_alignment(pad, offset, M, N, K):
    for out in (F16, F32):
        check(M, N, K, F16, out=out, pad=pad, offset=offset, seed=pad)
    check(M, N, K, E4M3, pad=pad, offset=offset, seed=pad)


@pytest.mark.parametrize("path", ["tile", "split", "few"])
@pytest.mark.parametrize("M,N,K", [(13, 40, 264), (16, 100, 512), (150, 72, 1000), (333, 168, 136)])
def test_small_integers_are_exact(path, M, N, K, tune):
    if path == "few" and M > 16:
        pytest.skip("up to 16 tokens")
    tune.setenv("TPGEMM_LINEAR_PATH", path)
    g = torch.Generator(device="cuda").manual_seed(M)
    A = torch.randint(-2, 3, (M, K), generator=g, device="cuda")
    W = torch.randint(-2, 3, (2 * N, K), generator=g, device="cuda")
    b = torch.randint(-9, 10, (2 * N,), generator=g, device="cuda")
    z = A.double() @ W.double().t() + b.double()
    for act in ("none", "relu"):  # sums below 2^12 in size, products below 2^24: every value is exact
        pre = torch.empty(M, 2 * N, device="cuda")
        y = tp.gated_linear(A.bfloat16(), W.bfloat16(), b.float(), act=act, out_dtype=F32, pre=pre)
        assert torch.equal(pre.double(), z)
        assert torch.equal(y.double(), (z[:, :N].clamp_min(0) if act == "relu" else z[:, :N]) * z[:, N:])


def test_empty():
    W = torch.ones(16, 8, device="cuda").half()
    assert tp.gated_linear(torch.ones(0, 8, device="cuda").half(), W).shape == (0, 8)
    assert tp.gated_linear(torch.ones(4, 8, device="cuda").half(), W[:0]).shape == (4, 0)
    b = torch.arange(16, device="cuda").half()
    for M in (3, 40):  # no K: the bias alone
        y = tp.gated_linear(torch.ones(M, 0, device="cuda").half(), W[:, :0], b, act="none")
        assert torch.equal(y, (b[:8] * b[8:]).expand(M, 8))


@pytest.mark.parametrize("M", [4, 40, 400])
def test_infinities_and_nan_stay_in_their_outputs(M):
    g = torch.Generator(device="cuda").manual_seed(M)
    A, W = view(g, M, 128, BF16), view(g, 144, 128, BF16)
    clean = tp.gated_linear(A, W)
    W[5, 3] = float("nan")        # gate 5
    W[72 + 9, 0] = float("inf")   # factor 9
    y = tp.gated_linear(A, W)
    assert torch.isnan(y[:, 5]).all()
    assert (torch.isinf(y[:, 9]) | torch.isnan(y[:, 9])).all()
    keep = [i for i in range(72) if i not in (5, 9)]
    assert torch.equal(y[:, keep], clean[:, keep])


def test_captured_and_on_another_stream():
    g = torch.Generator(device="cuda").manual_seed(3)
    A, W = view(g, 40, 264, BF16, 3), view(g, 200, 264, BF16)
    want = tp.gated_linear(A, W)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tp.gated_linear(A, W, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    dY, pre = view(g, 40, 100, BF16), view(g, 40, 200, BF16)
    grads = tp.gated_linear_backward(dY, A, W, pre)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tp.gated_linear(A, W)
        d = tp.gated_linear_backward(dY, A, W, pre)
    for _ in range(2):
        A.copy_(view(g, 40, 264, BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, tp.gated_linear(A, W))
        for a, b in zip(d, tp.gated_linear_backward(dY, A, W, pre)):
            assert torch.equal(a, b)
    assert torch.equal(d[2], grads[2])


# ---------------------------------------------------------------- gradients
def check_backward(M, N, K, dtype=BF16, act="silu", grad=None, pad=0, offset=0, seed=0, need=(True, True, True)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    grad = grad or dtype
    dY, pre = view(g, M, N, dtype, pad, offset), view(g, M, 2 * N, dtype, pad, offset, 1.5)
    A, W = view(g, M, K, dtype, pad, offset), view(g, 2 * N, K, dtype, pad, offset, N ** -0.5)
    got = tp.gated_linear_backward(dY, A, W, pre, act=act, grad_dtype=grad, need=need)
    want, bound = more.gated_backward(dY, A, W, pre, act, grad)
    for name, a, v, b, kind, asked in zip(("dA", "dW", "dbias"), got, want, bound, (dtype, grad, grad), need):
        if not asked:
            assert a is None
            continue
        assert a.dtype is kind and a.shape == v.shape
        ok, why = ref.within(a, v, b)
        assert ok, f"{name}: {why}"


@pytest.mark.parametrize("M,N,K", SIZES)
def test_backward_sizes(M, N, K):
    check_backward(M, N, K, seed=M)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("grad", [F16, BF16, F32])
def test_backward_types(dtype, act, grad):
    for M, N, K in ((3, 72, 256), (100, 33, 65), (700, 264, 128)):
        check_backward(M, N, K, dtype, act, grad, seed=M)


@pytest.mark.parametrize("dtype,std", [(BF16, 1.0), (F16, 1.0), (F16, 1e-6), (BF16, 1e-20)])
@pytest.mark.parametrize("M,N,K", [(100, 72, 264), (700, 264, 136)])
def test_32_bit_weight_gradients_see_all_of_dz(dtype, std, M, N, K):
    # dz as a rounding and its rest: within 2^-18 of bf16's and 2^-24 of f16's terms (whose rest is
    # kept away from f16's subnormal numbers), with a few roundings of its own, and two sums over M
    g = torch.Generator(device="cuda").manual_seed(M)
    pre, A, W = view(g, M, 2 * N, dtype), view(g, M, K, dtype), view(g, 2 * N, K, dtype)
    dY = view(g, M, N, dtype, std=std)
    _, dW, db = tp.gated_linear_backward(dY, A, W, pre, act="none", grad_dtype=F32)
    dz = torch.cat([dY.double() * pre[:, N:].double(), dY.double() * pre[:, :N].double()], 1)
    terms = dz.abs().t() @ A.double().abs()
    want = dz.t() @ A.double()
    ok, why = ref.within(dW, want, (2.0 ** -17 + 2 * ref.acc(M)) * terms + 2.0 ** -22 * want.abs() + 1e-44)
    assert ok, why
    assert float((dW.double() - want).norm() / want.norm()) <= 1e-5


@pytest.mark.parametrize("M,N,K", [(40, 200, 9000), (300, 264, 16384)])
def test_long_sums_of_32_bit_outputs(M, N, K):
    # two sums of random signs in each output, in pieces: off by less than 1e-5 of the outputs' size
    g = torch.Generator(device="cuda").manual_seed(K)
    A, W = view(g, M, K, BF16), view(g, 2 * N, K, BF16, std=K ** -0.5)
    y = tp.gated_linear(A, W, act="none", out_dtype=F32)
    z = A.double() @ W.double().t()
    want = z[:, :N] * z[:, N:]
    assert float((y.double() - want).norm() / want.norm()) <= 1e-5


@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (1, 0), (0, 1), (8, 4)])
def test_backward_strides(pad, offset):
    for M, N, K in ((3, 72, 256), (60, 100, 264), (300, 264, 96)):
        check_backward(M, N, K, F16, pad=pad, offset=offset, seed=pad)


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True), (False, False, False)])
def test_backward_of_some(need):
    for M in (30, 700):
        check_backward(M, 72, 96, need=need, act="gelu")


def test_backward_empty():
    W = torch.ones(16, 8, device="cuda").half()
    z = lambda *s: torch.zeros(*s, device="cuda").half()  # noqa: E731
    dA, dW, db = tp.gated_linear_backward(z(0, 8), z(0, 8), W, z(0, 16))
    assert dA.shape == (0, 8) and (dW == 0).all() and (db == 0).all() and dW.shape == (16, 8)
    dA, dW, db = tp.gated_linear_backward(z(4, 0), z(4, 8), W[:0], z(4, 0))
    assert (dA == 0).all() and dA.shape == (4, 8) and dW.shape == (0, 8) and db.shape == (0,)
    dA, dW, db = tp.gated_linear_backward(z(4, 8) + 1, z(4, 0), W[:, :0], z(4, 16) + 1, act="none")
    assert dA.shape == (4, 0) and dW.shape == (16, 0) and (db == 4).all()


@pytest.mark.parametrize("act", ref.ACTS)
def test_gradients_against_differences(act):
    # L = sum(c y) by the formula in 64 bits, moved by t along a direction v of each argument: the slope
    # (L(t) - L(-t)) / 2t is off by t^2 / 6 of the third derivative, at most c (2 |u| |dg|^3 + 3 dg^2 |du|)
    # where z moves by (dg, du) (act's third derivative is at most 2, its second 1). Small whole arguments
    # and halves make the stored z exact, and keep the gates off relu's bend. What the kernel's gradients
    # may be off by is their bound.
    g = torch.Generator(device="cuda").manual_seed(5)
    M, N, K = 20, 24, 8
    A = torch.randint(-1, 2, (M, K), generator=g, device="cuda").bfloat16()
    W = torch.randint(-1, 2, (2 * N, K), generator=g, device="cuda").bfloat16()
    b = torch.randint(-1, 2, (2 * N,), generator=g, device="cuda") + 0.5
    c = view(g, M, N, BF16)
    z = A.double() @ W.double().t() + b.double()
    pre = z.bfloat16()
    assert torch.equal(pre.double(), z)

    def loss(A, W, b):
        z = A @ W.t() + b
        return float((ref.act(z[:, :N], act) * z[:, N:] * c.double()).sum())
    got = tp.gated_linear_backward(c, A, W, pre, act=act, grad_dtype=F32)
    _, bounds = more.gated_backward(c, A, W, pre, act, F32)
    args, t = [A.double(), W.double(), b.double()], 2.0 ** -10
    for i, (grad, bound) in enumerate(zip(got, bounds)):
        v = torch.randn(args[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + t * v, args[i] - t * v
        slope = (loss(*up) - loss(*down)) / (2 * t)
        dz = (v @ args[1].t() if i == 0 else args[0] @ v.t() if i == 1 else v.expand(M, 2 * N)).abs()
        dg, du = dz.chunk(2, 1)
        third = float((c.double().abs() * (2 * z[:, N:].abs() * dg ** 3 + 3 * dg ** 2 * du)).sum())
        off = float((bound * v.abs()).sum()) + t * t / 6 * third + 1e-9
        assert abs(slope - float((grad.double() * v).sum())) <= off, act
