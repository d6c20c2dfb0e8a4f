"""The layer norm and its gradients where blocks walk many rows (GPU only): rows that start anywhere,
whole rows whose team is no power of two, several teams to a block and several rows to a team, with
residual, dropout and the gradient past the norm, padded and in place."""
import pytest
import torch

import test_layernorm_gpu as ln
import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
# Rows of any width, more than one to an SM: one warp to a row, several, a block.
ANYWHERE = [(5000, 37), (3000, 523), (333, 1001), (2000, 1501), (2000, 2101), (1000, 4099), (400, 9001), (320, 16383)]
# Whole pieces of 16 bytes, in teams of 96 to 480 threads (and of a row's last few).
WHOLE = [(153, 2560), (1300, 2560), (400, 5120), (400, 6144), (320, 7168), (320, 12288)]
ALIGNED = [(1300, 264), (1300, 1032), (700, 2568), (400, 9000)]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("rows,cols", ANYWHERE + WHOLE + ALIGNED)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_norm(rows, cols, dtype):
    ln.check(rows, cols, dtype, True, ln.NUMBERS, wdtype=F32 if dtype is F16 else None, seed=cols)
    ln.check(rows, cols, dtype, rows % 2 == 0, None, "row" if dtype is BF16 else None, seed=cols + 1, bias=False)


@pytest.mark.parametrize("rows,cols", ANYWHERE + WHOLE + ALIGNED)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_gradients(rows, cols, dtype):
    ln.check_backward(rows, cols, dtype, True, ln.NUMBERS, F32, wdtype=F32 if dtype is F16 else None, seed=cols)
    ln.check_backward(rows, cols, dtype, False, None, seed=cols + 1)


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (7, 3), (8, 4)])
@pytest.mark.parametrize("rows,cols", [(2500, 40), (2500, 1024), (2100, 1501), (400, 5120)])
def test_padded(rows, cols, pad, offset):
    for dtype in (F16, F32):
        ln.check(rows, cols, dtype, True, ln.NUMBERS, pad=pad, offset=offset, seed=pad)
        ln.check_backward(rows, cols, dtype, True, ln.NUMBERS, pad=pad, offset=offset, seed=pad)


@pytest.mark.parametrize("rows,cols", [(5000, 37), (2000, 1001), (2000, 1501), (1000, 4099), (400, 5120), (320, 9001)])
def test_in_place(rows, cols):
    # a team's rows to come are on their way while it writes; what it writes is another row's neighbour
    g = ln.gen(cols)
    x, r, e = (ln.normal(g, rows, cols, dtype=BF16) for _ in range(3))
    w, b = ln.normal(g, cols, dtype=BF16), ln.normal(g, cols, dtype=BF16)
    d = tp.Dropout(*ln.NUMBERS)
    n = tp.layernorm(x, w, b, r, dropout=d, need_stats=True)
    for which in (0, 1):
        a = [x.clone(), r.clone()]
        m = tp.layernorm(a[0], w, b, a[1], dropout=d, out_h=a[which])
        assert torch.equal(m.y, n.y) and torch.equal(a[which], n.h)
    y = x.clone()
    tp.layernorm(y, w, b, out=y)
    assert torch.equal(y, tp.layernorm(x, w, b).y)
    want = tp.layernorm_backward(x, n.h, n.mean, n.rstd, w, e, dropout=d)
    for which in range(3):
        a = [x.clone(), n.h.clone(), e.clone()]
        got = tp.layernorm_backward(a[0], a[1], n.mean, n.rstd, w, a[2], dropout=d, out=a[which])
        assert all(torch.equal(i, j) for i, j in zip(got, want))


@pytest.mark.parametrize("rows,cols", [(3000, 523), (1000, 4099), (400, 5120)])
def test_repeats(rows, cols):
    g = ln.gen(cols)
    x, r = ln.normal(g, rows, cols, dtype=BF16), ln.normal(g, rows, cols, dtype=BF16)
    w = ln.normal(g, cols, dtype=BF16)
    d = tp.Dropout(*ln.NUMBERS)
    n = tp.layernorm(x, w, w, r, dropout=d, need_stats=True)
    first = tp.layernorm_backward(x, n.h, n.mean, n.rstd, w, r, dropout=d, grad_dtype=F32)
    for _ in range(3):
        m = tp.layernorm(x, w, w, r, dropout=d, need_stats=True)
        assert all(torch.equal(i, j) for i, j in zip(m, n) if i is not None)
        again = tp.layernorm_backward(x, n.h, n.mean, n.rstd, w, r, dropout=d, grad_dtype=F32)
        assert all(torch.equal(i, j) for i, j in zip(again, first))
