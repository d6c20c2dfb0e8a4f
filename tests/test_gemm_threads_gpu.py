"""The multiply and the vectorised copy called by two host threads at once (GPU only), on problems whose
plans give one kernel different amounts of shared memory, which one thread must not set for the
other's launch."""
import ctypes

import pytest
import torch

import test_more_ops_threads_gpu as threads
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


@pytest.mark.parametrize("one,other", [
    ((512, 512, 256, 0), (2048, 2048, 1024, 0)), ((512, 512, 256, 1), (2048, 2048, 1024, 1)),
    ((1024, 1024, 512, 0), (1024, 1024, 512, 1)), ((144, 4104, 264, 0), (64, 4096, 512, 1))])
def test_two_threads_in_the_library(one, other):
    lib, made = tp.library(), []
    for M, N, K, beta in (one, other):
        stream = torch.cuda.Stream()
        A, B, C = threads.normal(M, K), threads.normal(N, K), threads.normal(M, N, dtype=torch.float32)
        D = torch.empty(M, N, device="cuda")
        args = (D.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr() if beta else None, M, N, K, 0, 1,
                tp.TPGEMM_BF16, float(beta), stream.cuda_stream)
        made.append((args, D, (A, B, C, stream)))
    for args, _, _ in made:
        assert lib.tpgemm_gemm(*args) == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()
    torch.cuda.synchronize()
    want = [D.clone() for _, D, _ in made]

    def work(i):
        for _ in range(5000):
            assert lib.tpgemm_gemm(*made[i][0]) == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()
    wrong = threads.at_once(work)
    assert not wrong, wrong
    assert all(torch.equal(D, w) for (_, D, _), w in zip(made, want))


def test_two_threads_copy():
    lib, made = tp.library(), []
    for rows in (48, 200):
        d, stream = tp.vcopy_desc(rows, 256, 4, threads=256), torch.cuda.Stream()
        src, n = threads.normal(rows, 256, dtype=torch.float32), rows * 1024
        dst = torch.empty_like(src)
        made.append(((dst.data_ptr(), src.data_ptr(), n, ctypes.byref(d), 1, 0, None, stream.cuda_stream), dst, src, d, stream))
    torch.cuda.synchronize()

    def work(i):
        for _ in range(5000):
            assert lib.tpgemm_vcopy_roundtrip(*made[i][0]) == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()
    wrong = threads.at_once(work)
    assert not wrong, wrong
    assert all(torch.equal(dst, src) for _, dst, src, _, _ in made)
