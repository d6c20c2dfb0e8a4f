"""Products of small integers, which 32-bit sums hold exactly (GPU only): each kernel of the linear
layer and of its gradients, at any length of the sum, has to give every bit."""
import pytest
import torch

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


def ints(g, *shape, dtype, ld=None):
    """Whole numbers from -3 to 3 (sums of 2^20 of their products stay below 2^24), rows ld apart."""
    ld = shape[1] if ld is None else ld
    buf = torch.randint(-3, 4, (shape[0], ld), generator=g, device="cuda").to(dtype)
    return buf[:, : shape[1]]


def check(M, N, K, dtype, g, lda=None, ldw=None):
    A, W = ints(g, M, K, dtype=dtype, ld=lda), ints(g, N, K, dtype=dtype, ld=ldw)
    b, r = ints(g, 1, N, dtype=F32)[0], ints(g, M, N, dtype=F32)
    z = torch.empty(M, N, device="cuda")
    want = A.double() @ W.double().t()
    assert torch.equal(tp.linear(A, W, out_dtype=F32).double(), want)
    assert torch.equal(tp.linear(A, W, b, r, act="relu", out_dtype=F32, pre=z).double(),
                       (want + b).clamp_min(0) + r)
    assert torch.equal(z.double(), want + b)


@pytest.mark.parametrize("K", [1, 63, 64, 65, 513, 4104, 20001])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3, E5M2])
@pytest.mark.parametrize("M,N", [(1, 200), (9, 33), (16, 1000), (17, 130), (144, 520), (260, 136), (300, 1000)])
def test_as_planned(M, N, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(K + M)
    check(M, N, K, dtype, g)
    check(M, N, K, dtype, g, lda=K + 3, ldw=K + 5)


@pytest.mark.parametrize("path,bn,split", [("tile", 32, 0), ("tile", 160, 0), ("tile", 224, 0), ("tile", 256, 0),
                                           ("split", 0, 1), ("split", 0, 2), ("split", 0, 4), ("split", 0, 8)])
@pytest.mark.parametrize("M,N,K", [(40, 520, 1032), (300, 136, 1040), (520, 776, 4104)])
def test_each_kernel(path, bn, split, M, N, K, tune):
    g = torch.Generator(device="cuda").manual_seed(bn + split)
    tune.setenv("TPGEMM_LINEAR_PATH", path)
    if bn:
        tune.setenv("TPGEMM_LINEAR_BN", str(bn))
    if split:
        tune.setenv("TPGEMM_LINEAR_SPLIT", str(split))
    for dtype in (BF16, E4M3):
        check(M, N, K, dtype, g)


@pytest.mark.parametrize("M,N,K", [(1, 72, 200), (16, 264, 520), (100, 520, 264), (513, 200, 1040), (4100, 136, 136),
                                   (33, 1000, 1001)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradients(M, N, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(M)
    dY, A, W, Z = (ints(g, *s, dtype=dtype) for s in ((M, N), (M, K), (N, K), (M, N)))
    for act in ("none", "relu"):
        dz = dY.double() * (1 if act == "none" else (Z > 0))
        dA, dW, db = tp.linear_backward(dY, A, W, Z, act=act, grad_dtype=F32)
        assert torch.equal(dA, (dz @ W.double()).float().to(dtype))
        assert torch.equal(dW.double(), dz.t() @ A.double())
        assert torch.equal(db.double(), dz.sum(0))
