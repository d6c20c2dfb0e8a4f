"""The linear layer and its gradients against 64-bit formulas (GPU only): sizes from one token up,
odd sizes, every type and activation, strides and misaligned rows, in-place residuals, other
streams and graphs, offsets past 32 bits, and what infinities and NaN become."""
import math

import pytest
import torch

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def guarded(rows, cols, dtype, ld=None, offset=0):
    """A [rows, cols] view inside a buffer of NaN, and a check that nothing else was written."""
    ld = cols if ld is None else ld
    n = max(1, rows) * ld + 2 * 256 + offset
    buf = torch.full((n,), float("nan"), dtype=dtype, device="cuda")
    view = buf.as_strided((rows, cols), (ld, 1), 256 + offset)

    def check():
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep.as_strided((rows, cols), (ld, 1), 256 + offset).fill_(False)
        assert torch.isnan(buf.float())[keep].all(), "written outside the output"
    return view, check


def check_linear(M, N, K, dtype, act="none", bias=True, residual=True, pre=False, out=None,
                 scales=None, seed=0, lda=None, ldw=None, ldy=None, offset=0):
    g = gen(seed)
    fp8 = dtype in (E4M3, E5M2)
    out = out or (BF16 if fp8 else dtype)

    def operand(rows, std, ld):
        ld = K if ld is None else ld
        buf = normal(g, max(1, rows) * ld + offset, std=std, dtype=dtype)
        return buf.as_strided((rows, K), (ld, 1), offset)
    A = operand(M, 4.0 if fp8 else 1.0, lda)
    W = operand(N, 4.0 / math.sqrt(max(K, 1)) if not fp8 else 4.0, ldw)
    scales = fp8 if scales is None else scales
    sa = torch.rand(M, generator=g, device="cuda") / 4 if scales else None
    sw = torch.rand(N, generator=g, device="cuda") / math.sqrt(max(K, 1)) if scales else None
    b = normal(g, N, dtype=out) if bias else None
    r = normal(g, M, N, dtype=out) if residual else None
    y, y_ok = guarded(M, N, out, ldy, offset)
    z, z_ok = guarded(M, N, out, ldy, offset) if pre else (None, lambda: None)
    tp.linear(A, W, b, r, act=act, scale_a=sa, scale_w=sw, out=y, pre=z)
    torch.cuda.synchronize()
    y_ok(), z_ok()
    ry, rz, by, bz = ref.linear(A, W, b, r, act, sa, sw, out)
    ok, why = ref.within(y, ry, by)
    assert ok, why
    if pre:
        ok, why = ref.within(z, rz, bz)
        assert ok, "pre: " + why


SIZES = [(1, 1, 1), (1, 8, 16), (1, 4096, 4096), (2, 100, 72), (3, 257, 1001), (7, 1000, 520),
         (8, 24, 8192), (9, 136, 2000), (16, 512, 64), (16, 33, 4097), (17, 16, 16), (18, 130, 96),
         (31, 1000, 1000), (64, 2056, 1040), (77, 129, 333), (128, 128, 128), (129, 64, 264),
         (144, 1640, 4104), (255, 200, 72), (256, 256, 4096), (257, 1, 65), (300, 300, 300),
         (384, 1024, 72), (511, 513, 515), (512, 512, 2048), (1000, 24, 24), (1025, 2049, 136),
         (2048, 1536, 512)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
def test_sizes(M, N, K, dtype):
    check_linear(M, N, K, dtype, act="silu", pre=True, seed=M + N + K)


@pytest.mark.parametrize("M,N,K", [(1, 96, 160), (13, 200, 136), (100, 264, 200), (400, 520, 136)])
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype,out", [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F16), (E4M3, F16),
                                       (E5M2, BF16), (E5M2, F32), (E4M3, BF16)])
def test_types_and_activations(M, N, K, act, dtype, out):
    check_linear(M, N, K, dtype, act=act, pre=True, out=out, seed=M + len(act))


@pytest.mark.parametrize("M,N,K", [(1, 264, 512), (16, 264, 512), (40, 264, 512), (300, 264, 512)])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("pre", [False, True])
def test_each_part_of_the_epilogue(M, N, K, bias, residual, pre):
    check_linear(M, N, K, BF16, act="gelu", bias=bias, residual=residual, pre=pre, seed=7)
    check_linear(M, N, K, E4M3, bias=bias, residual=residual, pre=pre, scales=pre, seed=8)


@pytest.mark.parametrize("M,N,K", [(1, 72, 136), (12, 72, 136), (50, 72, 136), (260, 200, 136)])
@pytest.mark.parametrize("lda,ldw,ldy,offset", [
    (200, 152, 208, 0),  # rows 16-byte aligned
    (201, 153, 211, 0),  # odd row strides
    (200, 152, 208, 1),  # aligned strides from a misaligned start
    (None, None, None, 3),
    (136, 137, 208, 0),  # one operand of each kind
    (137, 136, 209, 8),
])
def test_strides_and_alignment(M, N, K, lda, ldw, ldy, offset):
    for dtype in (F16, E5M2):
        check_linear(M, N, K, dtype, act="relu", pre=True, lda=lda, ldw=ldw, ldy=ldy,
                     offset=offset, seed=M + offset)


@pytest.mark.parametrize("K", [1, 7, 8, 31, 64, 100, 129, 511, 1024, 3000, 16384, 20001])
@pytest.mark.parametrize("M", [1, 5, 16, 24, 200, 520])
def test_reduction_lengths(M, K):
    check_linear(M, 144, K, BF16, act="none", out=F32, seed=K)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_empty_sizes(M):
    # A reduction over nothing is zero; no rows or columns is no work.
    check_linear(M, 40, 0, F16, act="gelu", pre=True)
    W = torch.zeros(0, 16, dtype=F16, device="cuda")
    A = torch.zeros(M, 16, dtype=F16, device="cuda")
    assert tp.linear(A, W).shape == (M, 0)
    assert tp.linear(A[:0], A).shape == (0, M)


@pytest.mark.parametrize("M", [1, 16, 60, 300])
def test_residual_in_place_and_repeatable(M):
    g = gen(M)
    A, W = normal(g, M, 520, dtype=BF16), normal(g, 200, 520, std=0.05, dtype=BF16)
    r = normal(g, M, 200, dtype=BF16)
    y = tp.linear(A, W, None, r, act="silu")
    assert torch.equal(y, tp.linear(A, W, None, r, act="silu"))
    x = r.clone()
    tp.linear(A, W, None, x, act="silu", out=x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("M", [1, 16, 100, 300])
def test_other_stream_and_graph(M):
    g = gen(11)
    A, W = normal(g, M, 256, dtype=F16), normal(g, 512, 256, std=0.1, dtype=F16)
    want = tp.linear(A, W, act="gelu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.zeros(M, 512, dtype=F16, device="cuda")
    torch.cuda.synchronize()
    tp.linear(A, W, act="gelu", out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out2 = torch.zeros_like(out)
    with torch.cuda.graph(graph):
        tp.linear(A, W, act="gelu", out=out2)
        tp.linear(out2, W.t().contiguous(), residual=A, out=A)  # a chain that changes its input
    keep = A.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, want)
    assert not torch.equal(A, keep)


@pytest.mark.parametrize("M", [1, 9, 64, 280])
def test_infinities_and_nan(M):
    # A NaN of A fills its row; an infinity of W its column, with the sign of what it meets;
    # other outputs are what they are without them.
    g = gen(3)
    A, W = normal(g, M, 136, dtype=F16).abs() + 0.1, normal(g, 48, 136, dtype=F16)
    clean = tp.linear(A, W)
    A2, W2 = A.clone(), W.clone()
    A2[M - 1, 5] = float("nan")
    W2[7, 100] = float("inf")
    y = tp.linear(A2, W2)
    assert torch.isnan(y[M - 1]).all()
    assert (y[: M - 1, 7] == float("inf")).all()
    keep = [i for i in range(48) if i != 7]
    assert torch.equal(y[: M - 1][:, keep], clean[: M - 1][:, keep])
    # infinities in the residual pass through; a saturated activation stays finite
    r = torch.zeros(M, 48, dtype=F16, device="cuda")
    r[0, 0] = float("-inf")
    assert tp.linear(A, W, None, r)[0, 0] == float("-inf")
    big = torch.full((48,), -60000.0, dtype=F16, device="cuda")
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        assert (tp.linear(A, W, big, act=act) == 0).all()


@pytest.mark.parametrize("M", [2, 18, 260])
def test_offsets_past_32_bits(M):
    # Rows so far apart that an element's offset does not fit 32 bits.
    ld = (1 << 32) // (M - 1) + 8
    ld -= ld % 8
    buf = torch.empty((M - 1) * ld + 64, dtype=E5M2, device="cuda")
    A = buf.as_strided((M, 64), (ld, 1))
    A.copy_(normal(gen(5), M, 64).to(E5M2))
    W = normal(gen(6), 80, 64).to(E5M2)
    y = tp.linear(A, W)
    assert torch.equal(y, tp.linear(A.contiguous(), W))
    wide = torch.empty(((1 << 31) // (M - 1) // 8 * 8 + 8) * (M - 1) + 80, dtype=BF16, device="cuda")
    out = wide.as_strided((M, 80), (((1 << 31) // (M - 1) // 8 * 8 + 8), 1))
    tp.linear(A, W, out=out)
    assert torch.equal(out, y)


# ------------------------------------------------------------------ gradients
def check_backward(M, N, K, dtype, act, grad, seed=0, lds=None, need=(True, True, True)):
    g = gen(seed)

    def mat(rows, cols, i, std=1.0):
        ld = cols if lds is None else cols + lds[i]
        return normal(g, max(1, rows) * ld, std=std, dtype=dtype).as_strided((rows, cols), (ld, 1))
    dY, A = mat(M, N, 0), mat(M, K, 1)
    W, pre = mat(N, K, 2, 0.1), mat(M, N, 3, 2.0)
    got = tp.linear_backward(dY, A, W, pre, act=act, grad_dtype=grad, need=need)
    torch.cuda.synchronize()
    want, bound = ref.linear_backward(dY, A, W, pre, act, grad)
    for name, x, y, b, asked in zip(("dA", "dW", "dbias"), got, want, bound, need):
        assert (x is not None) == asked
        if asked:
            ok, why = ref.within(x, y, b)
            assert ok, f"{name}: {why}"


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 512, 256), (3, 65, 129), (16, 264, 520), (17, 8, 8),
                                   (33, 1000, 24), (100, 520, 264), (128, 256, 512), (129, 127, 1001),
                                   (256, 24, 640), (300, 300, 300), (513, 72, 1040), (1000, 520, 8),
                                   (2048, 512, 384), (4100, 136, 136)])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dtype,grad", [(F16, F16), (BF16, F32)])
def test_backward_sizes(M, N, K, act, dtype, grad):
    check_backward(M, N, K, dtype, act, grad, seed=M + N)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype,grad", [(F16, F32), (F16, BF16), (BF16, BF16), (BF16, F16)])
def test_backward_activations_and_types(act, dtype, grad):
    check_backward(72, 200, 136, dtype, act, grad, seed=1)
    check_backward(300, 136, 264, dtype, act, grad, seed=2)


@pytest.mark.parametrize("lds", [(8, 16, 24, 40), (1, 3, 5, 7), (0, 1, 0, 0), (1, 0, 0, 8), (0, 0, 1, 0)])
@pytest.mark.parametrize("M", [1, 24, 300])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_backward_strides(lds, M, act):
    check_backward(M, 136, 72, F16, act, F16, lds=lds, seed=M)


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True),
                                  (True, False, True), (False, False, False)])
def test_backward_of_what_is_wanted(need):
    check_backward(40, 72, 136, BF16, "silu", F32, need=need)
    check_backward(40, 72, 136, BF16, "none", F32, need=need)


def test_backward_of_nothing():
    z = lambda *s: torch.zeros(*s, dtype=F16, device="cuda")  # noqa: E731
    dA, dW, db = tp.linear_backward(z(0, 24), z(0, 40), z(24, 40), z(0, 24), act="silu")
    assert dA.shape == (0, 40) and (dW == 0).all() and (db == 0).all()
    dA, dW, db = tp.linear_backward(z(5, 0), z(5, 40), z(0, 40))
    assert (dA == 0).all() and dA.shape == (5, 40) and dW.shape == (0, 40)
    dA, dW, db = tp.linear_backward(z(5, 24) + 1, z(5, 0), z(24, 0))
    assert dA.shape == (5, 0) and (db == 5).all()


@pytest.mark.parametrize("act", ref.ACTS)
def test_backward_against_differences(act):
    # The directional derivative of L = sum(Y o G) along random directions, by central
    # differences of the 64-bit forward: the error is that of the gradients' own bounds plus the
    # differences' (1e-6 of the sum of |terms| at this step).
    g = gen(21)
    M, N, K = 24, 40, 56
    A, W = normal(g, M, K, dtype=BF16), normal(g, N, K, std=0.3, dtype=BF16)
    b = normal(g, N, dtype=BF16)
    G = normal(g, M, N, dtype=BF16)

    def z_of(a, w, c):
        return a @ w.t() + c
    # The pre-activation as the forward stores it, and the loss around that value.
    z0 = z_of(A.double(), W.double(), b.double())
    pre = z0.to(BF16)
    shift = pre.double() - z0
    dA, dW, db = tp.linear_backward(G, A, W, pre, act=act, grad_dtype=F32)
    (_, _, _), (bA, bW, bb) = ref.linear_backward(G, A, W, pre, act, F32)

    def loss(a, w, c):
        return (ref.act(z_of(a, w, c) + shift, act) * G.double()).sum()
    a, w, c = A.double(), W.double(), b.double()
    if act == "relu":  # keep away from the corner
        assert pre.double().abs().min() > 1e-4
    h = 1e-6
    for _ in range(4):
        va, vw, vc = (torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)
                      for t in (a, w, c))
        diff = (loss(a + h * va, w + h * vw, c + h * vc)
                - loss(a - h * va, w - h * vw, c - h * vc)) / (2 * h)
        got = (dA.double() * va).sum() + (dW.double() * vw).sum() + (db.double() * vc).sum()
        size = (dA.double() * va).abs().sum() + (dW.double() * vw).abs().sum() + 1
        slack = (bA * va.abs()).sum() + (bW * vw.abs()).sum() + (bb * vc.abs()).sum()
        assert abs(diff - got) <= slack + 1e-5 * size


def test_backward_repeats_bit_for_bit():
    g = gen(4)
    args = [normal(g, 700, 264, dtype=BF16), normal(g, 700, 136, dtype=BF16),
            normal(g, 264, 136, dtype=BF16), normal(g, 700, 264, dtype=BF16)]
    one = tp.linear_backward(*args, act="gelu_tanh", grad_dtype=F32)
    two = tp.linear_backward(*args, act="gelu_tanh", grad_dtype=F32)
    assert all(torch.equal(x, y) for x, y in zip(one, two))


def test_python_refusals():
    g = gen(0)
    A, W = normal(g, 4, 16, dtype=F16), normal(g, 8, 16, dtype=F16)
    r = torch.zeros(4, 8, dtype=F16, device="cuda")
    cases = [(TypeError, lambda: tp.linear(A, W.to(BF16))),
             (TypeError, lambda: tp.linear(A, W, r[0].float())),
             (TypeError, lambda: tp.linear(A, W, None, r.float())),
             (TypeError, lambda: tp.linear(A.double(), W.double())),
             (ValueError, lambda: tp.linear(A, W[:, :8])),
             (ValueError, lambda: tp.linear(A.t(), A.t())),
             (ValueError, lambda: tp.linear(A[:1].expand(4, 16), W)),
             (ValueError, lambda: tp.linear(A, W, r[0][:4])),
             (ValueError, lambda: tp.linear(A, W, None, r[:3])),
             (ValueError, lambda: tp.linear(A, W, act="swish")),
             (ValueError, lambda: tp.linear(A, W.cpu())),
             (tp.TpgemmError, lambda: tp.linear(A, W, out=A.as_strided((4, 8), (16, 1)))),
             (tp.TpgemmError, lambda: tp.linear(A, W, scale_a=torch.ones(4, device="cuda"))),
             (ValueError, lambda: tp.linear_backward(r, A, W, act="silu")),
             (ValueError, lambda: tp.linear_backward(r[:, :4], A, W)),
             (TypeError, lambda: tp.linear_backward(r, A, W, grad_dtype=torch.float64)),
             (ValueError, lambda: tp.rmsnorm(A, A[0], quant="block")),
             (ValueError, lambda: tp.rmsnorm(A, A[0], out_h=A)),
             (TypeError, lambda: tp.rmsnorm(A, A[0].to(BF16))),
             (tp.TpgemmError, lambda: tp.rmsnorm(A, A[0].clone(), eps=-1.0)),
             (tp.TpgemmError, lambda: tp.rmsnorm(A, A[0].clone(), quant="row", out_dtype=F16)),
             (ValueError, lambda: tp.rmsnorm_backward(A, A, A[0].float(), A[0].clone()))]
    for kind, call in cases:
        with pytest.raises(kind):
            call()


# Each kernel at sizes the planner would give to another, and the choices it makes within one.
@pytest.mark.parametrize("path", ["tile", "split"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (17, 16, 16), (129, 64, 264), (256, 256, 512),
                                   (300, 304, 304), (130, 1000, 72), (1000, 24, 24), (520, 776, 1032)])
def test_each_kernel(path, M, N, K, tune):
    tune.setenv("TPGEMM_LINEAR_PATH", path)
    for dtype in (BF16, E4M3):
        check_linear(M, N, K, dtype, act="silu", pre=True, seed=M + N + K)
    check_backward(M, N, K, F16, "gelu", F32, seed=M)
    tune.delenv("TPGEMM_LINEAR_PATH")


@pytest.mark.parametrize("bn", range(32, 257, 32))
def test_tile_widths(bn, tune):
    tune.setenv("TPGEMM_LINEAR_PATH", "tile")
    tune.setenv("TPGEMM_LINEAR_BN", str(bn))
    check_linear(1100, 1300, 520, BF16, act="silu", pre=bn % 64 == 0, seed=bn)
    check_linear(400, 520, 200, F16, act="gelu", seed=bn)
    check_linear(400, 520, 208, E4M3, act="gelu", seed=bn)
    check_backward(400, 200, 136, BF16, "none", BF16, seed=bn)
    for name in ("PATH", "BN"):
        tune.delenv("TPGEMM_LINEAR_" + name)


@pytest.mark.parametrize("split", range(1, 9))
@pytest.mark.parametrize("bp", [64, 80, 96, 112, 128])
def test_splits_and_tile_rows(split, bp, tune):
    tune.setenv("TPGEMM_LINEAR_PATH", "split")
    tune.setenv("TPGEMM_LINEAR_SPLIT", str(split))
    tune.setenv("TPGEMM_LINEAR_BP", str(bp))
    check_linear(40, 520, 1032, F16, act="gelu", pre=True, seed=bp)
    check_linear(300, 136, 1040, E4M3, act="gelu", seed=bp)
    if bp % 64 == 0:
        check_backward(24, 200, 328, BF16, "none", BF16, seed=bp)
        check_backward(520, 200, 136, BF16, "none", F32, seed=bp)
    for name in ("PATH", "SPLIT", "BP"):
        tune.delenv("TPGEMM_LINEAR_" + name)


def test_many_tiles_per_pair():
    # Several tiles to a pair of CTAs: both accumulators in turn, ragged on every side.
    check_linear(4100, 5000, 264, BF16, act="relu", pre=True, seed=1)
    check_linear(6000, 3000, 144, E5M2, act="none", seed=2)


@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 24, 3001), (8, 40, 128), (9, 17, 2000), (16, 1000, 520)])
def test_few_tokens_splits(split, M, N, K, tune):
    tune.setenv("TPGEMM_LINEAR_SPLIT", str(split))
    for dtype in (F16, BF16, E4M3, E5M2):
        check_linear(M, N, K, dtype, act="silu", pre=True, seed=split)
    tune.delenv("TPGEMM_LINEAR_SPLIT")


@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("M,N,K", [(200, 264, 8200), (264, 40, 8192), (24, 1000, 4104), (1000, 136, 9000)])
def test_splits_of_long_sums(split, M, N, K, tune):
    # Partial sums over the stages (long shares of K) and beside them, lines either way round.
    tune.setenv("TPGEMM_LINEAR_PATH", "split")
    tune.setenv("TPGEMM_LINEAR_SPLIT", str(split))
    check_linear(M, N, K, BF16, act="silu", pre=True, seed=split)
    check_linear(M, N, K // 16, F16, act="gelu", out=F32, seed=split)
    for name in ("PATH", "SPLIT"):
        tune.delenv("TPGEMM_LINEAR_" + name)


def test_scratch_belongs_to_the_stream_it_is_used_on():
    # Memory freed on the current stream is handed out again at once: what a call on another
    # stream still uses must not be among it.
    g = gen(31)
    dY, Z = normal(g, 2000, 1000, dtype=F16), normal(g, 2000, 1000, dtype=F16)
    A, W = normal(g, 2000, 1001, dtype=F16), normal(g, 1000, 1001, std=0.1, dtype=F16)
    want = tp.linear_backward(dY, A, W, Z, act="silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(20):
        got = tp.linear_backward(dY, A, W, Z, act="silu", stream=s)
        junk = [torch.full((n * 1000,), 255, dtype=torch.uint8, device="cuda") for n in (2000, 4000, 8000)]
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
        del junk


def ones(g, *shape, dtype):
    """Values of -1, 0 and 1: sums of up to 256 of their products are exact in every output type."""
    return torch.randint(-1, 2, shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("bn", [None] + list(range(32, 257, 32)))
def test_short_sums_of_many_tiles_are_exact(bn, tune):
    # Many tiles to a pair of CTAs, short sums and nothing but the output to store: each tile's
    # stores follow the last one's at once, with odd numbers of chunks to a warp at most widths.
    tune.setenv("TPGEMM_LINEAR_PATH", "tile")
    if bn:
        tune.setenv("TPGEMM_LINEAR_BN", str(bn))
    g = gen(bn or 0)
    for M, N, K in [(4096, 4096, 64), (2100, 8200, 128), (4100, 2072, 72)]:
        for dtype, out in [(F16, F16), (BF16, BF16), (E4M3, BF16), (BF16, F32)]:
            A, W = ones(g, M, K, dtype=dtype), ones(g, N, K, dtype=dtype)
            want = (A.float() @ W.float().t()).to(out)
            for _ in range(3):
                assert torch.equal(tp.linear(A, W, out_dtype=out), want)
    # the gradients' products, along the operands' rows
    dY, A, W = (ones(g, *s, dtype=F16) for s in ((64, 4096), (64, 4104), (4096, 4104)))
    want = (dY.float().t() @ A.float()).half()
    for _ in range(3):
        assert torch.equal(tp.linear_backward(dY, A, W, need=(False, True, False))[1], want)
    dY, W = ones(g, 4104, 72, dtype=BF16), ones(g, 72, 4096, dtype=BF16)
    want = (dY.float() @ W.float()).bfloat16()
    A = torch.zeros(4104, 4096, dtype=BF16, device="cuda")
    for _ in range(3):
        assert torch.equal(tp.linear_backward(dY, A, W, need=(True, False, False))[0], want)
