"""Dropout against a mask drawn on the host: every type, odd widths and strides, the residual, in
place, infinities and NaN under the mask, probabilities at their ends, a counter in device memory
that a captured graph reads anew, other streams (GPU only)."""
import pytest
import torch

import more_ops_reference as more
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


def view(seed, rows, cols, dtype, pad=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.randn(rows * (cols + pad) + offset, generator=g, device="cuda").to(dtype)
    return flat.as_strided((rows, cols), (cols + pad, 1), offset)


def check(rows, cols, dtype, numbers, residual=False, pad=0, offset=0):
    x = view(1, rows, cols, dtype, pad, offset)
    r = view(2, rows, cols, dtype, pad, offset) if residual else None
    buf = torch.full((rows * (cols + pad) + offset + 64,), 7.0, dtype=dtype, device="cuda")
    y = buf.as_strided((rows, cols), (cols + pad, 1), offset)
    tp.dropout(x, tp.Dropout(*numbers), r, out=y)
    want, err = more.drop(x, numbers)
    if residual:
        want = want + r.double()
        err = err + more.E32 * want.abs()
    ok, why = ref.within(y, want, more.rounded(err, want, dtype))
    assert ok, why
    if not residual:  # the mask itself, bit for bit
        assert torch.equal(y == 0, (want == 0) | (want.to(dtype) == 0))
    between = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    between.as_strided((rows, cols), (cols + pad, 1), offset).fill_(False)
    assert (buf[between] == 7).all()


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 3), (1, 8), (3, 5), (2, 64), (37, 1001), (300, 7),
                                       (5, 4096), (70001, 8), (3, 70004), (513, 1032)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_sizes(rows, cols, dtype, residual):
    check(rows, cols, dtype, (0.3, 0x123456789ABCDEF0, 77), residual)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (8, 4), (16, 8)])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_strides(pad, offset, dtype):
    check(9, 264, dtype, (0.5, 3, 2 ** 63 + 5), True, pad, offset)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -33, 1e-3, 0.5, 0.999, 1 - 2.0 ** -20])
@pytest.mark.parametrize("seed,offset", [(0, 0), (2 ** 64 - 1, 2 ** 64 - 1), (2 ** 32, 2 ** 32)])
def test_numbers_at_their_ends(p, seed, offset):
    check(40, 200, F32, (p, seed, offset))


def test_share_of_dropped_elements():
    # 2^22 independent draws: their share is within six standard deviations
    for p in (0.01, 0.1, 0.5):
        y = tp.dropout(torch.ones(2048, 2048, device="cuda"), tp.Dropout(p, 9, 1))
        share = float((y == 0).double().mean())
        assert abs(share - p) <= 6 * (p * (1 - p)) ** 0.5 / 2 ** 11


def test_dropped_infinities_are_zero_and_kept_ones_stay():
    x = torch.full((16, 64), float("inf"), device="cuda")
    x[:, 1::2] = float("nan")
    keep = more.kept(16, 64, 0.5, 5, 0).cuda()
    y = tp.dropout(x, tp.Dropout(0.5, 5))
    assert (y[~keep] == 0).all() and torch.isinf(y[:, ::2][keep[:, ::2]]).all()
    assert torch.isnan(y[:, 1::2][keep[:, 1::2]]).all()


@pytest.mark.parametrize("cols", [96, 101])
def test_in_place_and_backward(cols):
    x, r = view(3, 33, cols, BF16), view(4, 33, cols, BF16)
    d = tp.Dropout(0.25, 11, 12)
    want = tp.dropout(x, d, r)
    a, b = x.clone(), r.clone()
    assert torch.equal(tp.dropout(a, d, r, out=a), want) and torch.equal(tp.dropout(x, d, b, out=b), want)
    dy = view(5, 33, cols, BF16)
    dx = tp.dropout_backward(dy, d)
    ok, why = ref.within(dx, *(lambda v, e: (v, more.rounded(e, v, BF16)))(*more.drop(dy, (0.25, 11, 12))))
    assert ok, why


def test_strides_do_not_change_the_mask():
    x = torch.ones(20, 100, device="cuda")
    wide = torch.ones(20, 131, device="cuda")[:, 3:103]
    d = tp.Dropout(0.5, 1)
    assert torch.equal(tp.dropout(x, d), tp.dropout(wide, d))


def test_empty():
    x = torch.zeros(0, 64, device="cuda")
    assert tp.dropout(x, tp.Dropout(0.5, 1)).shape == (0, 64)
    assert tp.dropout(x.t(), tp.Dropout(0.5, 1)).shape == (64, 0)


def test_counter_in_memory_and_replays():
    x = torch.ones(64, 64, device="cuda")
    counter = torch.tensor([10], device="cuda")
    d = tp.Dropout(0.5, 42, counter)
    assert torch.equal(tp.dropout(x, d), tp.dropout(x, tp.Dropout(0.5, 42, 10)))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tp.dropout(x, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tp.dropout(x, d)
        counter.add_(1)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, tp.dropout(x, tp.Dropout(0.5, 42, 10 + i)))
    assert int(counter) == 13


@pytest.mark.parametrize("bad", [dict(p=1.0), dict(p=-0.1), dict(p=float("nan"))])
def test_refused_probabilities(bad):
    with pytest.raises(tp.TpgemmError):
        tp.dropout(torch.ones(2, 2, device="cuda"), tp.Dropout(seed=1, **bad))


def test_refused_arguments():
    x = torch.ones(4, 8, device="cuda")
    for d in (tp.Dropout(0.1, -1), tp.Dropout(0.1, 2 ** 64), tp.Dropout(0.1, 1, -1),
              tp.Dropout(0.1, 1, torch.tensor([1])), tp.Dropout(0.1, 1, torch.tensor([1, 2], device="cuda"))):
        with pytest.raises(ValueError):
            tp.dropout(x, d)
    with pytest.raises(TypeError):
        tp.dropout(x, tp.Dropout(0.1, 1, 0.5))
    with pytest.raises(tp.TpgemmError):  # an output that overlaps x by halves
        flat = torch.ones(40, device="cuda")
        tp.dropout(flat[:32].view(4, 8), tp.Dropout(0.1, 1), out=flat[4:36].view(4, 8))
