"""The root-mean-square norm and its gradients against 64-bit formulas (GPU only): rows from one
token up, odd widths, every type, both kinds of 8-bit scales, strides, in-place use, zero rows,
infinities and NaN, and the path into the two multiplies that read its 8-bit output."""
import pytest
import torch

import ops_reference as ref
import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
SIZES = [(1, 1), (1, 7), (1, 8192), (2, 31), (3, 32), (5, 33), (4, 64), (9, 100), (17, 1000),
         (33, 1001), (300, 128), (64, 1024), (7, 1032), (40, 2048), (20, 4096), (6, 4104), (3, 5000),
         (5, 8192), (2, 16384), (2, 16392), (3, 20000), (2, 32768), (2, 33000), (1, 70001)]


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


def normal(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def view(g, rows, cols, dtype, pad=0, offset=0, std=1.0):
    ld = cols + pad
    return normal(g, rows * ld + offset, std=std, dtype=dtype).as_strided((rows, cols), (ld, 1),
                                                                         offset)


def check(rows, cols, dtype, residual, quant=None, out=None, wdtype=None, pad=0, offset=0, seed=0,
          std=1.0, eps=1e-5):
    g = gen(seed)
    x = view(g, rows, cols, dtype, pad, offset, std)
    r = view(g, rows, cols, dtype, pad, offset, std) if residual else None
    w = (1 + normal(g, cols, std=0.2)).to(wdtype or dtype)
    kind = out or (dtype if quant is None else E4M3)
    buf = torch.full((rows * (cols + pad) + offset + 64,), 1.0, device="cuda").to(kind)
    y = buf.as_strided((rows, cols), (cols + pad, 1), offset)
    n = tp.rmsnorm(x, w, r, eps=eps, quant=quant, out=y, need_rstd=True)
    torch.cuda.synchronize()
    # what lies between and after the rows is untouched
    mask = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    mask.as_strided((rows, cols), (cols + pad, 1), offset).fill_(False)
    assert (buf.float()[mask] == 1).all()
    ry, rh, rr = ref.rmsnorm(x, w, r, eps)
    # a 32-bit sum of squares, a square root and a division: relative error below
    e = ref.acc(8 * cols) / 2 + 2.0 ** -21
    ok, why = ref.within(n.rstd, rr, e * rr)
    assert ok, "rstd: " + why
    if residual:
        ok, why = ref.within(n.h, rh, (ref.U[dtype] + 2.0 ** -23) * rh.abs() + ref.TINY[dtype])
        assert ok, "h: " + why
    else:
        assert n.h is None
    err = (e + 2.0 ** -21) * ry.abs()
    if quant is None:
        ok, why = ref.within(n.y, ry, err + ref.U[kind] * ry.abs() + ref.TINY[kind])
        assert ok, "y: " + why
        return
    top, emax = ref.FP8[kind][:2]
    if quant == "row":
        want = (ry.abs().amax(1) / top).clamp_min(2.0 ** -126)
        ok, why = ref.within(n.scale, want, 2 * (e + 2.0 ** -21) * want)
        assert ok, "scale: " + why
        scale = n.scale.double()[:, None].expand(rows, cols)
    else:
        assert n.scale.shape == (rows, (cols + 31) // 32) and n.scale.dtype is torch.uint8
        pad_y = torch.nn.functional.pad(ry, (0, -cols % 32)).unflatten(1, (-1, 32))
        amax = pad_y.abs().amax(2)
        # the exponent is exact unless amax lies within the error of a power of two
        lo = torch.floor(torch.log2((amax * (1 - 2 * e)).clamp_min(1e-300))) - emax
        hi = torch.floor(torch.log2((amax * (1 + 2 * e)).clamp_min(1e-300))) - emax
        code = n.scale.double() - 127
        assert ((code >= lo.clamp(-127, 127)) & (code <= hi.clamp(-127, 127))).all()
        scale = torch.exp2(code).repeat_interleave(32, 1)[:, :cols]
    # each code is a nearest value of the type: within half a spacing of y / scale, saturating
    q = n.y.double()
    v = (ry / scale).clamp(-top, top)
    half = torch.maximum(ref.quantum(v, kind), ref.quantum(q, kind)) / 2
    ok, why = ref.within(q, v, half * (1 + 2.0 ** -10) + 4 * err / scale)
    assert ok, "codes: " + why


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("quant", [None, "row", "mx"])
@pytest.mark.parametrize("residual", [False, True])
def test_sizes(rows, cols, quant, residual):
    check(rows, cols, BF16, residual, quant, seed=rows + cols)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("wdtype", [None, F32])
@pytest.mark.parametrize("quant,out", [(None, F16), (None, BF16), (None, F32), ("row", E4M3),
                                       ("row", E5M2), ("mx", E4M3), ("mx", E5M2)])
def test_types(dtype, wdtype, quant, out):
    for rows, cols in ((5, 264), (3, 1001), (40, 4096)):
        check(rows, cols, dtype, True, quant, out, wdtype, seed=cols)


@pytest.mark.parametrize("pad,offset", [(8, 0), (24, 8), (16, 16), (1, 0), (0, 1), (7, 3), (8, 4)])
@pytest.mark.parametrize("cols", [96, 1000, 2056, 9000])
@pytest.mark.parametrize("quant", [None, "row", "mx"])
def test_strides_and_alignment(pad, offset, cols, quant):
    for dtype in (F16, F32):
        check(6, cols, dtype, True, quant, pad=pad, offset=offset, seed=pad)


def test_many_rows():
    check(70000, 8, F16, True, "row", seed=1)
    check(5000, 520, BF16, True, "mx", seed=2)


@pytest.mark.parametrize("std", [1e-30, 1e-12, 1e4, 1e15])
@pytest.mark.parametrize("quant", [None, "row", "mx"])
def test_extreme_magnitudes(std, quant):
    # eps = 0: the norm undoes any magnitude whose squares stay within 32 bits
    eps = 0.0 if std >= 1e-12 else 1e-30
    check(4, 1024, F32, False, quant, out=None if quant else F32, std=std, eps=eps, seed=3)


@pytest.mark.parametrize("cols", [40, 1001, 4096, 40000])
@pytest.mark.parametrize("quant", ["row", "mx"])
@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_zero_rows_infinities_and_nan(cols, quant, kind):
    x = normal(gen(9), 5, cols, dtype=BF16)
    x[0] = 0
    x[2, cols // 2] = float("inf")
    x[3, 0] = float("nan")
    w = torch.ones(cols, dtype=BF16, device="cuda")
    n = tp.rmsnorm(x, w, quant=quant, out_dtype=kind)
    clean = tp.rmsnorm(x[[1, 4]].contiguous(), w, quant=quant, out_dtype=kind)
    value = n.y.float() * n.scale[:, None] if quant == "row" else ref.decode_mx(n.y, n.scale)
    assert (value[0] == 0).all()
    assert torch.isnan(value[3]).all()
    # an infinity makes rstd zero: the element itself is 0 * inf, a NaN, and poisons its scale
    blk = slice(0, cols) if quant == "row" else slice(cols // 64 * 32, min(cols, cols // 64 * 32 + 32))
    assert torch.isnan(value[2, blk]).all()
    assert torch.equal(n.y[[1, 4]].view(torch.uint8), clean.y.view(torch.uint8))
    assert torch.equal(n.scale[[1, 4]], clean.scale)
    # an infinity in the weight: y itself is infinite and its scale NaN
    w2 = w.clone()
    w2[1] = float("inf")
    m = tp.rmsnorm(x[[1]].contiguous(), w2, quant=quant, out_dtype=kind)
    value = m.y.float() * m.scale[:, None] if quant == "row" else ref.decode_mx(m.y, m.scale)
    assert torch.isnan(value[0, : (cols if quant == "row" else 32)]).all()


@pytest.mark.parametrize("cols", [100, 1024, 4096, 50000])
def test_in_place(cols):
    g = gen(1)
    x, r = normal(g, 9, cols, dtype=BF16), normal(g, 9, cols, dtype=BF16)
    w = normal(g, cols, dtype=BF16)
    n = tp.rmsnorm(x, w, r)
    r2 = r.clone()
    m = tp.rmsnorm(x, w, r2, out_h=r2)
    assert torch.equal(m.y, n.y) and torch.equal(r2, n.h)
    x2 = x.clone()
    m = tp.rmsnorm(x2, w, r, out_h=x2)
    assert torch.equal(m.y, n.y) and torch.equal(x2, n.h)
    x3 = x.clone()
    tp.rmsnorm(x3, w, out=x3)
    assert torch.equal(x3, tp.rmsnorm(x, w).y)


def test_no_rows():
    x = torch.zeros(0, 64, dtype=F16, device="cuda")
    w = torch.ones(64, dtype=F16, device="cuda")
    assert tp.rmsnorm(x, w, x, quant="mx").scale.shape == (0, 2)
    dx, dw = tp.rmsnorm_backward(x, x, torch.zeros(0, device="cuda"), w)
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_row_scales_feed_linear():
    g = gen(2)
    x, r = normal(g, 24, 520, dtype=BF16), normal(g, 24, 520, dtype=BF16)
    w = 1 + normal(g, 520, std=0.1, dtype=BF16)
    W = normal(g, 96, 520, std=16.0).to(E4M3)
    sw = torch.rand(96, generator=g, device="cuda") / 300
    n = tp.rmsnorm(x, w, r, quant="row")
    y = tp.linear(n.y, W, scale_a=n.scale, scale_w=sw, out_dtype=F32)
    want = (n.y.double() * n.scale.double()[:, None]) @ (W.double() * sw.double()[:, None]).t()
    ok, why = ref.within(y, want, ref.acc(520) * 2 * want.abs().max() + 1e-3)
    assert ok, why


def test_mx_scales_feed_the_block_scaled_multiply():
    g = gen(3)
    x = normal(g, 64, 512, dtype=BF16)
    w = 1 + normal(g, 512, std=0.1, dtype=BF16)
    n = tp.rmsnorm(x, w, quant="mx")
    B = normal(g, 128, 512).to(E4M3)
    sb = torch.full((128, 16), 127, dtype=torch.uint8, device="cuda")
    y = tp.gemm_mx(n.y, B, n.scale, sb)
    a = ref.decode_mx(n.y, n.scale)
    ok, why = ref.within(y, a @ B.double().t(), ref.acc(512) * (a.abs() @ B.double().abs().t()))
    assert ok, why


# ------------------------------------------------------------------ gradients
def check_grad(rows, cols, dtype, dh, grad=None, wdtype=None, pad=0, offset=0, seed=0,
               need=(True, True)):
    g = gen(seed)
    dy = view(g, rows, cols, dtype, pad, offset)
    h = view(g, rows, cols, dtype, pad, offset, std=2.0)
    d = view(g, rows, cols, dtype, pad, offset) if dh else None
    w = (1 + normal(g, cols, std=0.2)).to(wdtype or dtype)
    rstd = 1 / torch.sqrt(h.float().square().mean(1) + 1e-5)
    grad = grad or dtype
    dx, dw = tp.rmsnorm_backward(dy, h, rstd, w, d, grad_dtype=grad, need=need)
    torch.cuda.synchronize()
    (rx, rw), (bx, bw) = ref.rmsnorm_backward(dy, h, rstd, w, d)
    if need[0]:
        ok, why = ref.within(dx, rx, bx + ref.U[dtype] * rx.abs() + ref.TINY[dtype])
        assert ok, "dx: " + why
    if need[1]:
        ok, why = ref.within(dw, rw, bw + ref.U[grad] * rw.abs() + ref.TINY[grad])
        assert ok, "dweight: " + why
    assert (dx is not None, dw is not None) == tuple(need)


@pytest.mark.parametrize("rows,cols", SIZES + [(2000, 72), (1000, 1024), (700, 4096), (333, 1001)])
@pytest.mark.parametrize("dh", [False, True])
def test_grad_sizes(rows, cols, dh):
    check_grad(rows, cols, BF16, dh, seed=rows)
    check_grad(rows, cols, F16, dh, grad=F32, seed=cols)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("grad", [F16, BF16, F32])
@pytest.mark.parametrize("wdtype", [None, F32])
def test_grad_types(dtype, grad, wdtype):
    check_grad(50, 520, dtype, True, grad, wdtype)
    check_grad(20, 1003, dtype, False, grad, wdtype)


@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 16), (1, 0), (0, 1), (8, 4)])
@pytest.mark.parametrize("cols", [96, 2056, 9000])
def test_grad_strides(pad, offset, cols):
    for dtype in (F16, F32):
        check_grad(30, cols, dtype, True, pad=pad, offset=offset)


@pytest.mark.parametrize("need", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("cols", [264, 40000])
def test_grad_of_what_is_wanted(need, cols):
    check_grad(20, cols, BF16, True, need=need)


@pytest.mark.parametrize("cols", [264, 1001, 8192, 40000])
def test_grad_in_place_and_repeatable(cols):
    g = gen(8)
    dy, h, dh = (normal(g, 40, cols, dtype=BF16) for _ in range(3))
    w = normal(g, cols, dtype=BF16)
    rstd = 1 / torch.sqrt(h.float().square().mean(1))
    dx, dw = tp.rmsnorm_backward(dy, h, rstd, w, dh)
    for i in range(3):
        args = [dy.clone(), h.clone(), dh.clone()]
        x, v = tp.rmsnorm_backward(args[0], args[1], rstd, w, args[2], out=args[i])
        assert torch.equal(x, dx) and torch.equal(v, dw) and x.data_ptr() == args[i].data_ptr()


def test_grad_against_differences():
    # Central differences of the 64-bit forward along random directions, the weights in the loss
    # those of dy and of dh; 32-bit tensors, so the gradients' own error is near 1e-6 of the terms.
    g = gen(31)
    rows, cols, eps = 12, 200, 1e-5
    x, w = normal(g, rows, cols), 1 + normal(g, cols, std=0.3)
    dy, dh = normal(g, rows, cols), normal(g, rows, cols)

    def loss(a, b):
        y, h, _ = ref.rmsnorm(a, b, None, eps)
        return (y * dy.double()).sum() + (h * dh.double()).sum()
    rstd = tp.rmsnorm(x, w, eps=eps, need_rstd=True).rstd
    dx, dw = tp.rmsnorm_backward(dy, x, rstd, w, dh)
    a, b, step = x.double(), w.double(), 1e-6
    for _ in range(4):
        va = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float64)
        vb = torch.randn(cols, generator=g, device="cuda", dtype=torch.float64)
        diff = (loss(a + step * va, b + step * vb) - loss(a - step * va, b - step * vb)) / (2 * step)
        got = (dx.double() * va).sum() + (dw.double() * vb).sum()
        size = (dx.double() * va).abs().sum() + (dw.double() * vb).abs().sum()
        assert abs(diff - got) <= 2e-6 * size + 1e-4


def test_streams_and_graph():
    g = gen(5)
    x, r = normal(g, 40, 2048, dtype=BF16), normal(g, 40, 2048, dtype=BF16)
    w = normal(g, 2048, dtype=BF16)
    want = tp.rmsnorm(x, w, r, quant="row")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = tp.rmsnorm(x, w, r, quant="row")
    s.synchronize()
    assert torch.equal(got.y.view(torch.uint8), want.y.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = tp.rmsnorm(x, w, r, quant="row")
        tp.rmsnorm_backward(x, r, again.scale, w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again.h, want.h) and torch.equal(again.scale, want.scale)


def test_offsets_past_32_bits():
    rows, ld = 3, (1 << 31) + 16
    buf = torch.empty(rows * ld, dtype=BF16, device="cuda")
    x = buf.as_strided((rows, 1000), (ld, 1))
    x.copy_(normal(gen(2), rows, 1000))
    w = torch.ones(1000, dtype=BF16, device="cuda")
    assert torch.equal(tp.rmsnorm(x, w).y, tp.rmsnorm(x.contiguous(), w).y)
    rstd = tp.rmsnorm(x, w, need_rstd=True).rstd
    a = tp.rmsnorm_backward(x, x, rstd, w)
    b = tp.rmsnorm_backward(x.contiguous(), x.contiguous(), rstd, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("cols", [1, 32, 333, 512, 1001, 2048, 4096, 8192, 16384, 20000])
@pytest.mark.parametrize("eps", [0.0, 1e-8, 1e-6, 1e-3])
@pytest.mark.parametrize("rows", [3, 400])
def test_mx_scale_at_a_power_of_two(cols, eps, rows):
    # Rows of +-1 under a weight of 2: |y| = 2 / sqrt(1 + eps), which is 2 or less than it by as
    # little as 5e-9 of it, less than 32-bit arithmetic tells apart. The exponent is exact.
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 0.5, -1.0, 1.0).bfloat16()
    w = torch.full((cols,), 2.0, device="cuda").bfloat16()
    r = tp.rmsnorm(x, w, eps=eps, quant="mx")
    code = 127 - 8 + (1 if eps == 0 else 0)
    assert (r.scale == code).all()
    top = 256.0 if eps == 0 else 448.0  # 2 / 2^-7; just under 2 / 2^-8, past the largest
    assert torch.equal(r.y.float(), x.float() * top)
    half = torch.zeros_like(x)
    both = tp.rmsnorm(x, w, half, eps=eps, quant="mx", out_h=x)  # h in place of x
    assert torch.equal(both.y.view(torch.uint8), r.y.view(torch.uint8))
    assert torch.equal(both.scale, r.scale)
