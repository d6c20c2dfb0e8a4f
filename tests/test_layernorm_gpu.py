"""The layer norm and its gradients against 64-bit formulas (GPU only): rows from one token up, odd
widths, every type, row scales, dropout and residual, strides, in-place use, large means, infinities
and NaN, and the path into the 8-bit linear layer."""
import pytest
import torch

import more_ops_reference as more
import ops_reference as ref
import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
SIZES = [(1, 1), (1, 7), (1, 8192), (2, 31), (3, 32), (5, 33), (4, 64), (9, 100), (17, 1000),
         (33, 1001), (300, 128), (64, 1024), (7, 1032), (40, 2048), (400, 4096), (6, 4104), (3, 5000),
         (5, 8192), (2, 16384), (2, 16392), (3, 20000), (2, 32768), (2, 33000), (1, 70001)]
NUMBERS = (0.25, 0xFEDCBA9876543210, 2 ** 33 + 9)


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, mean=0.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def view(g, rows, cols, dtype, pad=0, offset=0, std=1.0, mean=0.0):
    ld = cols + pad
    return normal(g, rows * ld + offset, std=std, mean=mean, dtype=dtype).as_strided((rows, cols), (ld, 1), offset)


def check(rows, cols, dtype, residual=False, numbers=None, quant=None, out=None, wdtype=None, pad=0,
          offset=0, seed=0, std=1.0, mean=0.5, eps=1e-5, bias=True):
    g = gen(seed)
    x = view(g, rows, cols, dtype, pad, offset, std, mean)
    r = view(g, rows, cols, dtype, pad, offset, std, mean) if residual else None
    w = (1 + normal(g, cols, std=0.2)).to(wdtype or dtype)
    b = normal(g, cols, std=0.3, dtype=wdtype or dtype) if bias else None
    kind = out or (dtype if quant is None else E4M3)
    buf = torch.full((rows * (cols + pad) + offset + 64,), 1.0, device="cuda").to(kind)
    y = buf.as_strided((rows, cols), (cols + pad, 1), offset)
    n = tp.layernorm(x, w, b, r, eps=eps, dropout=None if numbers is None else tp.Dropout(*numbers),
                     quant=quant, out=y, need_stats=True)
    torch.cuda.synchronize()
    mask = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    mask.as_strided((rows, cols), (cols + pad, 1), offset).fill_(False)
    assert (buf.float()[mask] == 1).all()
    (ry, rh, rm, rr), (ey, eh, em, er) = more.layernorm(x, w, b, r, eps, numbers)
    for name, got, want, err in (("mean", n.mean, rm, em), ("rstd", n.rstd, rr, er)):
        ok, why = ref.within(got, want, more.rounded(err, want, F32))
        assert ok, name + ": " + why
    if residual or numbers:
        ok, why = ref.within(n.h, rh, more.rounded(eh, rh, dtype))
        assert ok, "h: " + why
    else:
        assert n.h is None
    if quant is None:
        ok, why = ref.within(n.y, ry, more.rounded(ey, ry, kind))
        assert ok, "y: " + why
        return
    top = ref.FP8[kind][0]
    want = (ry.abs().amax(1) / top).clamp_min(2.0 ** -126)
    ok, why = ref.within(n.scale, want, 1.01 * ey.amax(1) / top + 4 * more.E32 * want)
    assert ok, "scale: " + why
    scale = n.scale.double()[:, None]
    # each code is a nearest value of the type: within half a spacing of y / scale, saturating
    q, v = n.y.double(), (ry / scale).clamp(-top, top)
    half = torch.maximum(ref.quantum(v, kind), ref.quantum(q, kind)) / 2
    ok, why = ref.within(q, v, half * (1 + 2.0 ** -10) + 2 * ey / scale)
    assert ok, "codes: " + why


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("quant", [None, "row"])
@pytest.mark.parametrize("residual,numbers", [(False, None), (True, None), (True, NUMBERS), (False, NUMBERS)])
def test_sizes(rows, cols, quant, residual, numbers):
    check(rows, cols, BF16, residual, numbers, quant, seed=rows + cols)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("wdtype", [None, F32])
@pytest.mark.parametrize("quant,out", [(None, F16), (None, BF16), (None, F32), ("row", E4M3), ("row", E5M2)])
def test_types(dtype, wdtype, quant, out):
    for rows, cols in ((5, 264), (3, 1001), (40, 4096), (2, 17000)):
        check(rows, cols, dtype, True, NUMBERS, quant, out, wdtype, seed=cols, bias=cols != 264)


@pytest.mark.parametrize("pad,offset", [(8, 0), (24, 8), (16, 16), (1, 0), (0, 1), (7, 3), (8, 4)])
@pytest.mark.parametrize("cols", [96, 1000, 2056, 9000, 17000])
def test_strides_and_alignment(pad, offset, cols):
    for dtype in (F16, F32):
        check(6, cols, dtype, True, NUMBERS, pad=pad, offset=offset, seed=pad)
        check(6, cols, dtype, True, None, "row", pad=pad, offset=offset, seed=pad)


def test_many_rows():
    check(70000, 8, F16, True, NUMBERS, seed=1)
    check(5000, 520, BF16, True, None, "row", seed=2)


@pytest.mark.parametrize("std,mean", [(1e-12, 0.0), (1e10, 0.0), (1.0, 1000.0), (0.01, 300.0), (1e-3, -1.0)])
@pytest.mark.parametrize("cols", [100, 1024, 4099, 20000])
def test_magnitudes_and_means(std, mean, cols):
    check(4, cols, F32, std=std, mean=mean, eps=0.0 if std != 1e-3 else 1e-6, seed=3)


def test_rows_of_one_value():
    # var is 0 and y the bias, but for what the mean is off by
    for cols in (1, 40, 4096, 17001):
        for value in (3.0, -0.1, 0.0, 1e4):
            check(3, cols, F32, std=0.0, mean=value)


@pytest.mark.parametrize("cols", [40, 1001, 4096, 40000])
@pytest.mark.parametrize("quant", [None, "row"])
def test_infinities_and_nan_stay_in_their_rows(cols, quant):
    x = normal(gen(9), 5, cols, dtype=BF16)
    x[0] = 0
    x[2, cols // 2] = float("inf")
    x[3, 0] = float("nan")
    w = torch.ones(cols, dtype=BF16, device="cuda")
    n = tp.layernorm(x, w, quant=quant)
    clean = tp.layernorm(x[[0, 1, 4]].contiguous(), w, quant=quant)
    value = n.y.float() * n.scale[:, None] if quant else n.y.float()
    assert torch.isnan(value[2:4]).all() and (value[0] == 0).all()
    assert torch.equal(n.y[[0, 1, 4]].float(), clean.y.float())


def test_what_dropout_removes_does_not_reach_the_row():
    keep = more.kept(8, 200, 0.5, 3, 0).cuda()
    x = torch.where(keep, normal(gen(4), 8, 200), torch.tensor(float("nan"), device="cuda"))
    w, b = torch.ones(200, device="cuda"), torch.zeros(200, device="cuda")
    d = tp.Dropout(0.5, 3)
    n = tp.layernorm(x, w, b, dropout=d)
    m = tp.layernorm(torch.where(keep, x, torch.zeros_like(x)), w, b, dropout=d)
    assert torch.equal(n.y, m.y) and torch.equal(n.h, m.h)


@pytest.mark.parametrize("cols", [100, 101, 1024, 4096, 50000])
def test_in_place(cols):
    g = gen(1)
    x, r = normal(g, 9, cols, dtype=BF16), normal(g, 9, cols, dtype=BF16)
    w, b = normal(g, cols, dtype=BF16), normal(g, cols, dtype=BF16)
    d = tp.Dropout(0.1, 1)
    n = tp.layernorm(x, w, b, r, dropout=d)
    for which in (0, 1):
        a = [x.clone(), r.clone()]
        m = tp.layernorm(a[0], w, b, a[1], dropout=d, out_h=a[which])
        assert torch.equal(m.y, n.y) and torch.equal(a[which], n.h)
    x3 = x.clone()
    tp.layernorm(x3, w, b, out=x3)
    assert torch.equal(x3, tp.layernorm(x, w, b).y)


def test_no_rows():
    x = torch.zeros(0, 64, dtype=F16, device="cuda")
    w = torch.ones(64, dtype=F16, device="cuda")
    assert tp.layernorm(x, w, w, x, quant="row").scale.shape == (0,)
    d = tp.layernorm_backward(x, x, torch.zeros(0, device="cuda"), torch.zeros(0, device="cuda"), w)
    assert d.dx.shape == (0, 64) and (d.dweight == 0).all() and (d.dbias == 0).all()


def test_row_scales_feed_linear():
    g = gen(2)
    x, w = normal(g, 24, 520, dtype=BF16), 1 + normal(g, 520, std=0.1, dtype=BF16)
    W = normal(g, 96, 520, std=16.0).to(E4M3)
    n = tp.layernorm(x, w, quant="row")
    y = tp.linear(n.y, W, scale_a=n.scale, out_dtype=F32)
    a = n.y.double() * n.scale.double()[:, None]
    ok, why = ref.within(y, a @ W.double().t(), ref.acc(520) * (a.abs() @ W.double().abs().t()) + 1e-30)
    assert ok, why


# ---------------------------------------------------------------- gradients
def check_backward(rows, cols, dtype, dh=False, numbers=None, grad=None, wdtype=None, pad=0, offset=0, seed=0,
                   need=(True, True, True, True)):
    g = gen(seed)
    dy, h = view(g, rows, cols, dtype, pad, offset), view(g, rows, cols, dtype, pad, offset, 2.0, 1.0)
    e = view(g, rows, cols, dtype, pad, offset) if dh else None
    w = (1 + normal(g, cols, std=0.2)).to(wdtype or dtype)
    mean = h.double().mean(1)
    rstd = (1 / torch.sqrt((h.double() - mean[:, None]).square().mean(1) + 1e-5)).float()
    mean = mean.float()
    grad = grad or w.dtype
    drop = None if numbers is None else tp.Dropout(*numbers)
    got = tp.layernorm_backward(dy, h, mean, rstd, w, e, dropout=drop, grad_dtype=grad, need=need)
    want, bound = more.layernorm_backward(dy, h, mean, rstd, w, e, numbers)
    for name, a, v, b, kind, asked in zip(got._fields, got, want, bound, (dtype, dtype, grad, grad), need):
        if not asked:
            assert a is None
            continue
        assert a.dtype is kind
        ok, why = ref.within(a, v, more.rounded(b, v, kind))
        assert ok, f"{name}: {why}"


@pytest.mark.parametrize("rows,cols", SIZES + [(1000, 64), (3000, 520), (700, 1024), (400, 8192), (320, 16384)])
@pytest.mark.parametrize("dh,numbers", [(False, None), (True, NUMBERS)])
def test_backward_sizes(rows, cols, dh, numbers):
    check_backward(rows, cols, BF16, dh, numbers, seed=rows + cols)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("wdtype", [None, F32])
@pytest.mark.parametrize("grad", [F16, BF16, F32])
def test_backward_types(dtype, wdtype, grad):
    for rows, cols in ((5, 264), (3, 1001), (40, 4096), (33, 9000), (2, 17000)):
        check_backward(rows, cols, dtype, True, NUMBERS, grad, wdtype, seed=cols)


@pytest.mark.parametrize("pad,offset", [(8, 0), (24, 8), (1, 0), (0, 1), (8, 4)])
@pytest.mark.parametrize("cols", [96, 1000, 2056, 9000, 17000])
def test_backward_strides(pad, offset, cols):
    for dtype in (F16, F32):
        check_backward(6, cols, dtype, True, NUMBERS, pad=pad, offset=offset, seed=pad)


@pytest.mark.parametrize("need", [(True, False, False, False), (False, True, False, False), (True, True, False, True),
                                  (False, False, True, True), (False, False, True, False), (False, False, False, True),
                                  (False, False, False, False)])
@pytest.mark.parametrize("numbers", [None, NUMBERS])
def test_backward_of_some(need, numbers):
    for cols in (100, 2048, 17000):
        check_backward(30, cols, BF16, True, numbers, need=need)


@pytest.mark.parametrize("cols", [100, 1024, 4099, 8192, 50000])
@pytest.mark.parametrize("numbers", [None, NUMBERS])
def test_backward_in_place(cols, numbers):
    g = gen(5)
    dy, h, e = (normal(g, 9, cols, dtype=BF16) for _ in range(3))
    w = normal(g, cols, dtype=BF16)
    mean, rstd = h.float().mean(1), torch.rand(9, generator=g, device="cuda") + 0.5
    d = None if numbers is None else tp.Dropout(*numbers)
    want = tp.layernorm_backward(dy, h, mean, rstd, w, e, dropout=d)
    for which in range(3):
        a = [dy.clone(), h.clone(), e.clone()]
        got = tp.layernorm_backward(a[0], a[1], mean, rstd, w, a[2], dropout=d, out=a[which])
        assert torch.equal(a[which], want.dx)
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_backward_repeats():
    g = gen(6)
    dy, h = normal(g, 999, 1000, dtype=BF16), normal(g, 999, 1000, dtype=BF16)
    mean, rstd, w = h.float().mean(1), torch.ones(999, device="cuda"), normal(g, 1000, dtype=BF16)
    first = tp.layernorm_backward(dy, h, mean, rstd, w, grad_dtype=F32)
    for _ in range(3):
        for a, b in zip(first, tp.layernorm_backward(dy, h, mean, rstd, w, grad_dtype=F32)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("rows,cols", [(3, 40), (5, 1001)])
def test_gradients_against_differences(rows, cols):
    # L = sum(c y + e h) of the kernel's own forward pass, moved by t along a direction of each
    # argument: (L(t) - L(-t)) / 2t is off by t^2 / 6 of the third derivative (arguments of size 1,
    # t = 2^-6: 4e-5 of the terms' size) and by the 32-bit roundings of L's terms over t (2^-20 of
    # their size, summed).
    g = gen(7)
    x, r, c, e = (normal(g, rows, cols) for _ in range(4))
    w, b = 1 + normal(g, cols, std=0.1), normal(g, cols)
    d = tp.Dropout(0.3, 8, 9)

    def loss(x, r, w, b):
        n = tp.layernorm(x, w, b, r, dropout=d, eps=1e-5)
        return float((n.y.double() * c.double() + n.h.double() * e.double()).sum())
    n = tp.layernorm(x, w, b, r, dropout=d, eps=1e-5, need_stats=True)
    got = tp.layernorm_backward(c, n.h, n.mean, n.rstd, w, e, dropout=d)
    args, t = [x, r, w, b], 2.0 ** -6
    for i, grad in enumerate((got.dx, got.dresidual, got.dweight, got.dbias)):
        v = normal(g, *args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + t * v, args[i] - t * v
        slope = (loss(*up) - loss(*down)) / (2 * t)
        size = float((grad.double() * v.double()).norm()) + (rows * cols) ** 0.5
        assert abs(slope - float((grad.double() * v.double()).sum())) <= 1e-3 * size
