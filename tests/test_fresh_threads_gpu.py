"""Entries called from a host thread that has made no CUDA call before (GPU only): such a thread has no
current context, which the driver's tensor-map encoder wants. torch's allocator may answer from
what it holds, so a Python call's first CUDA call can be the library's."""
import ctypes
import threading

import pytest
import torch

import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

M, N, K = 300, 256, 128


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


def in_a_fresh_thread(work):
    got = []
    t = threading.Thread(target=lambda: got.append(work()))
    t.start()
    t.join()
    torch.cuda.synchronize()
    return got[0]


def normal(*shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(sum(shape)), device="cuda").bfloat16()


@pytest.mark.parametrize("path", ["tile", "split"])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_layers(gated, path, tune):
    tune.setenv("TPGEMM_LINEAR_PATH", path)
    A, W = normal(M, K), normal(2 * N if gated else N, K)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    code = tp.TPGEMM_ELEM_BF16
    d = tp.LinearDesc(M, N, K, 0, 0, 0, 0, 0, code, code, tp.TPGEMM_ACT_SILU)
    torch.cuda.synchronize()
    lib = tp.library()
    fn = lib.tpgemm_gated_linear if gated else lib.tpgemm_linear
    args = (Y.data_ptr(), None, A.data_ptr(), W.data_ptr(), None, None, None) + (() if gated else (None,)) + \
        (ctypes.byref(d), None, 0, None)
    status, why = in_a_fresh_thread(lambda: (fn(*args), tp.tpgemm_last_error_detail()))
    assert status == tp.TPGEMM_OK, why
    assert torch.equal(Y, tp.gated_linear(A, W, act="silu") if gated else tp.linear(A, W, act="silu"))


def test_multiply():
    A, B = normal(256, K), normal(N, K)
    D = torch.empty(256, N, device="cuda")
    torch.cuda.synchronize()
    args = (D.data_ptr(), A.data_ptr(), B.data_ptr(), None, 256, N, K, 0, 1, tp.TPGEMM_BF16, 0.0, None)
    status, why = in_a_fresh_thread(lambda: (tp.library().tpgemm_gemm(*args), tp.tpgemm_last_error_detail()))
    assert status == tp.TPGEMM_OK, why
    assert torch.equal(D, tp.gemm(A, B, transB=True))


def test_norms_and_dropout():
    x, w = normal(M, K), normal(K)
    y = torch.empty_like(x)
    code = tp.TPGEMM_ELEM_BF16
    d, n = tp.DropoutDesc(M, K, 0, 0, 0, code, 0.1, 1, 2), tp.LayerNormDesc(M, K, 0, 0, 0, 0, code, code, code, 0, 1e-5)
    torch.cuda.synchronize()
    lib = tp.library()
    for fn, args, want in ((lib.tpgemm_dropout, (y.data_ptr(), x.data_ptr(), None, ctypes.byref(d), None),
                            lambda: tp.dropout(x, tp.Dropout(0.1, 1, 2))),
                           (lib.tpgemm_layernorm, (y.data_ptr(), None, None, None, None, x.data_ptr(), None, w.data_ptr(),
                                                   None, ctypes.byref(n), None), lambda: tp.layernorm(x, w).y)):
        status, why = in_a_fresh_thread(lambda: (fn(*args), tp.tpgemm_last_error_detail()))
        assert status == tp.TPGEMM_OK, why
        assert torch.equal(y, want())
