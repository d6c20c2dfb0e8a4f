"""The operators called by two host threads at once, each on a stream of its own (GPU only). The two
run the same kernel on sizes that want different amounts of shared memory, which one thread must not
set for the other's launch."""
import ctypes
import threading

import pytest
import torch

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


def normal(*shape, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def norm(rows, cols, wide):
    x, r, w = normal(rows, cols), normal(rows, cols), normal(cols, dtype=F32 if wide else BF16)
    return lambda: tp.layernorm(x, w, w, r).y


def norm_gradients(rows, cols, wide):
    dy, h, w = normal(rows, cols), normal(rows, cols), normal(cols, dtype=F32 if wide else BF16)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dh = dy if wide else None
    return lambda: tp.layernorm_backward(dy, h, mean, rstd, w, dh, grad_dtype=F32).dx


def gated(rows, cols, wide):
    A, W, pre = normal(rows, cols), normal(2 * cols, cols), normal(rows, 2 * cols)
    return lambda: tp.gated_linear_backward(tp.gated_linear(A, W), A, W, pre, grad_dtype=F32 if wide else BF16)[1]


def drop(rows, cols, wide):
    x = normal(rows, cols)
    return lambda: tp.dropout(x, tp.Dropout(0.1, 1, cols), x if wide else None)


def at_once(work):
    """work(i) in two threads that start together; what went wrong in them."""
    start, wrong = threading.Barrier(2), []

    def run(i):
        try:
            start.wait()
            work(i)
        except BaseException as e:  # (told by the caller)
            wrong.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return wrong


@pytest.mark.parametrize("make,one,other", [
    (norm, (8192, 4096), (400, 4096)), (norm, (200, 17000), (200, 50000)), (norm, (4000, 1501), (333, 1501)),
    (norm_gradients, (8192, 4096), (400, 4096)), (norm_gradients, (200, 17000), (200, 50000)),
    (norm_gradients, (4000, 4099), (333, 4099)), (gated, (40, 520), (700, 256)), (drop, (999, 1001), (64, 4096))])
def test_two_threads(make, one, other):
    calls = [make(*one, True), make(*other, False)]
    want = [call().clone() for call in calls]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(400):
                got = calls[i]()
            torch.cuda.current_stream().synchronize()
            assert torch.equal(got, want[i])
    wrong = at_once(work)
    assert not wrong, wrong


def entry(gradients, rows, cols, wide, stream):
    """A call of a C entry with all its arguments laid out, and what they point to."""
    lib, code = tp.library(), tp.TPGEMM_ELEM_F32 if wide else tp.TPGEMM_ELEM_BF16
    x, r, w = normal(rows, cols), normal(rows, cols), normal(cols, dtype=F32 if wide else BF16)
    y, h = torch.empty_like(x), torch.empty_like(x)
    if gradients:
        need = tp.tpgemm_layernorm_backward_workspace_bytes(rows, cols)
        ws, g, stats = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(2, cols, device="cuda"), \
            torch.ones(rows, device="cuda")
        d = tp.LayerNormGradDesc(rows, cols, 0, 0, 0, 0, 0, tp.TPGEMM_ELEM_BF16, code, tp.TPGEMM_ELEM_F32)
        fn, args = lib.tpgemm_layernorm_backward, (y.data_ptr(), None, g[0].data_ptr(), g[1].data_ptr(), x.data_ptr(),
                                                   r.data_ptr(), stats.data_ptr(), stats.data_ptr(), w.data_ptr(),
                                                   x.data_ptr() if wide else None, ctypes.byref(d), ws.data_ptr(), need, stream)
        return fn, args, (x, r, w, y, ws, g, stats, d)
    d = tp.LayerNormDesc(rows, cols, 0, 0, 0, 0, tp.TPGEMM_ELEM_BF16, code, tp.TPGEMM_ELEM_BF16, 0, 1e-5)
    fn, args = lib.tpgemm_layernorm, (y.data_ptr(), h.data_ptr(), None, None, None, x.data_ptr(), r.data_ptr(), w.data_ptr(),
                                      w.data_ptr(), ctypes.byref(d), stream)
    return fn, args, (x, r, w, y, h, d)


@pytest.mark.parametrize("gradients,one,other", [
    (False, (2000, 4096), (400, 4096)), (False, (160, 17000), (160, 50000)), (False, (2000, 1501), (333, 1501)),
    (True, (2000, 4096), (400, 4096)), (True, (1000, 4099), (333, 4099))])
def test_two_threads_in_the_library(gradients, one, other):
    # Nothing but the C entry in the threads' loops: two of them are in it for most of the time.
    streams = [torch.cuda.Stream() for _ in range(2)]
    made = [entry(gradients, *size, i == 0, streams[i].cuda_stream) for i, size in enumerate((one, other))]
    for fn, args, _ in made:
        assert fn(*args) == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()
    torch.cuda.synchronize()
    want = [keep[3].clone() for _, _, keep in made]

    def work(i):
        fn, args, _ = made[i]
        for _ in range(10000):
            assert fn(*args) == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()
    wrong = at_once(work)
    assert not wrong, wrong
    assert all(torch.equal(keep[3], y) for (_, _, keep), y in zip(made, want))
