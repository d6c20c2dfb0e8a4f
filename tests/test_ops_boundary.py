"""What the operators around the multiply refuse, without a GPU: every rejection names its reason
before anything is enqueued. Pointers are fake addresses that these paths never read."""
import pytest
import torch

import tile_primitive_tensor_gb300 as tp
from tile_primitive_tensor_gb300 import build as tpbuild

BASE = 0x7F0000000000
MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tpbuild.build()
    tp.library()


def addr(i, off=0):
    return BASE + 64 * MB * i + off


# Past validation a call fails for want of a GPU here, and on a GPU machine these addresses must not
# be launched on: accepted forms are only tried where there is no device.
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake addresses")


def linear(M=24, N=40, K=64, lda=0, ldw=0, ldr=0, ldy=0, ldz=0, dtype=tp.TPGEMM_ELEM_F16,
           out=tp.TPGEMM_ELEM_F16, act=0, Y=addr(0), Z=addr(1), A=addr(2), W=addr(3), sa=None, sw=None,
           bias=addr(4), R=addr(5), ws=None, wsb=0):
    d = tp.LinearDesc(M, N, K, lda, ldw, ldr, ldy, ldz, dtype, out, act)
    st = tp.tpgemm_linear(Y, Z, A, W, sa, sw, bias, R, d, ws, wsb, 0)
    return st, tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(M=-1), tp.TPGEMM_ERR_SHAPE, "M=-1"),
    (dict(N=1 << 30), tp.TPGEMM_ERR_SHAPE, "N=1073741824"),
    (dict(K=-5), tp.TPGEMM_ERR_SHAPE, "K=-5"),
    (dict(lda=63), tp.TPGEMM_ERR_SHAPE, "A: row stride 63"),
    (dict(ldw=1), tp.TPGEMM_ERR_SHAPE, "W: row stride 1"),
    (dict(ldr=-40), tp.TPGEMM_ERR_SHAPE, "R: row stride"),
    (dict(ldy=39), tp.TPGEMM_ERR_SHAPE, "Y: row stride"),
    (dict(ldz=8), tp.TPGEMM_ERR_SHAPE, "Z: row stride"),
    (dict(M=1 << 29, N=1 << 29), tp.TPGEMM_ERR_SHAPE, "memory"),
    (dict(dtype=tp.TPGEMM_E2M1), tp.TPGEMM_ERR_DTYPE, "dtype 4"),
    (dict(dtype=tp.TPGEMM_ELEM_F32), tp.TPGEMM_ERR_DTYPE, "dtype 8"),
    (dict(out=tp.TPGEMM_ELEM_E4M3), tp.TPGEMM_ERR_DTYPE, "out 2"),
    (dict(act=5), tp.TPGEMM_ERR_DTYPE, "activation 5"),
    (dict(act=-1), tp.TPGEMM_ERR_DTYPE, "activation -1"),
    (dict(sa=addr(6)), tp.TPGEMM_ERR_DTYPE, "e4m3 or e5m2"),
    (dict(Y=None), tp.TPGEMM_ERR_NULL, "Y is NULL"),
    (dict(A=None), tp.TPGEMM_ERR_NULL, "A is NULL"),
    (dict(W=None), tp.TPGEMM_ERR_NULL, "W is NULL"),
    (dict(Y=addr(0, 1)), tp.TPGEMM_ERR_ALIGN, "Y="),
    (dict(A=addr(2, 1)), tp.TPGEMM_ERR_ALIGN, "A="),
    (dict(bias=addr(4, 1)), tp.TPGEMM_ERR_ALIGN, "bias="),
    (dict(dtype=tp.TPGEMM_ELEM_E4M3, sw=addr(6, 2)), tp.TPGEMM_ERR_ALIGN, "scale_w="),
    (dict(Z=addr(0, 16)), tp.TPGEMM_ERR_ALIAS, "Y overlaps Z"),
    (dict(A=addr(0, 24 * 40 * 2 - 2)), tp.TPGEMM_ERR_ALIAS, "Y overlaps A"),
    (dict(R=addr(0, 2)), tp.TPGEMM_ERR_ALIAS, "Y overlaps R"),
    (dict(R=addr(0), ldr=48), tp.TPGEMM_ERR_ALIAS, "Y overlaps R"),
    (dict(Z=addr(5)), tp.TPGEMM_ERR_ALIAS, "Z overlaps R"),
    (dict(bias=addr(1)), tp.TPGEMM_ERR_ALIAS, "Z overlaps bias"),
    # slices of one buffer, rows of one pitch, that share columns
    (dict(ldy=200, A=addr(0, 2 * 39), lda=200), tp.TPGEMM_ERR_ALIAS, "Y overlaps A"),
    (dict(ldy=200, A=addr(0, 2 * 150), lda=200), tp.TPGEMM_ERR_ALIAS, "Y overlaps A"),
])
def test_linear_refuses(kw, status, frag):
    st, why = linear(**kw)
    assert st == status and frag in why, (st, why)


@needs_no_gpu
@pytest.mark.parametrize("kw", [
    dict(), dict(Z=None, bias=None, R=None), dict(R=addr(0)), dict(R=addr(0), ldr=48, ldy=48),
    dict(ldy=200, A=addr(0, 2 * 40), lda=200),  # side by side in one buffer
    dict(K=0, A=None, W=None), dict(M=1, lda=3000000), dict(A=addr(2, 2)),
    dict(dtype=tp.TPGEMM_ELEM_E5M2, A=addr(2, 1), sa=addr(6), sw=addr(7), out=8),
])
def test_linear_accepts(kw):
    need = tp.tpgemm_linear_workspace_bytes(
        kw.get("A", addr(2)), kw.get("W", addr(3)),
        tp.LinearDesc(24, 40, kw.get("K", 64), kw.get("lda", 0), 0, 0, 0, 0, kw.get("dtype", 0), 0, 0))
    st, why = linear(**kw, ws=addr(9) if need else None, wsb=need)
    assert st == tp.TPGEMM_ERR_ARCH, (st, why)


def test_linear_with_no_outputs_is_no_work():
    assert linear(M=0, Y=None, A=None)[0] == tp.TPGEMM_OK
    assert linear(N=0, Y=None, W=None)[0] == tp.TPGEMM_OK


def backward(M=24, N=40, K=64, dtype=0, grad=8, act=tp.TPGEMM_ACT_SILU, dA=addr(0), dW=addr(1),
             db=addr(2), dY=addr(3), A=addr(4), W=addr(5), Z=addr(6), ws=addr(9), wsb=None, **lds):
    d = tp.LinearGradDesc(M, N, K, *[lds.get(n, 0) for n in ("lddy", "ldz", "lda", "ldw", "ldda", "lddw")],
                          dtype, grad, act)
    if wsb is None:
        wsb = tp.tpgemm_linear_backward_workspace_bytes(dY, A, W, d)
    st = tp.tpgemm_linear_backward(dA, dW, db, dY, A, W, Z, d, ws, wsb, 0)
    return st, tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(M=-1), tp.TPGEMM_ERR_SHAPE, "M=-1"),
    (dict(dtype=tp.TPGEMM_ELEM_E4M3), tp.TPGEMM_ERR_DTYPE, "f16 or bf16"),
    (dict(grad=tp.TPGEMM_ELEM_E5M2), tp.TPGEMM_ERR_DTYPE, "grad 3"),
    (dict(act=9), tp.TPGEMM_ERR_DTYPE, "activation 9"),
    (dict(dY=None), tp.TPGEMM_ERR_NULL, "dY is NULL"),
    (dict(A=None), tp.TPGEMM_ERR_NULL, "A is NULL"),
    (dict(W=None), tp.TPGEMM_ERR_NULL, "W is NULL"),
    (dict(Z=None), tp.TPGEMM_ERR_NULL, "Z is NULL"),
    (dict(lddw=63), tp.TPGEMM_ERR_SHAPE, "dW: row stride 63"),
    (dict(dW=addr(1, 2)), tp.TPGEMM_ERR_ALIGN, "dW="),
    (dict(dA=addr(4)), tp.TPGEMM_ERR_ALIAS, "dA overlaps A"),
    (dict(dW=addr(5)), tp.TPGEMM_ERR_ALIAS, "dW overlaps W"),
    (dict(db=addr(1, 128)), tp.TPGEMM_ERR_ALIAS, "dW overlaps dbias"),
    (dict(ws=None), tp.TPGEMM_ERR_NULL, "workspace is NULL"),
    (dict(ws=addr(9, 128)), tp.TPGEMM_ERR_ALIGN, "256-byte"),
    (dict(wsb=512), tp.TPGEMM_ERR_NULL, "workspace of 512 bytes"),
    (dict(ws=addr(3)), tp.TPGEMM_ERR_ALIAS, "workspace overlaps dY"),
])
def test_linear_backward_refuses(kw, status, frag):
    st, why = backward(**kw)
    assert st == status and frag in why, (st, why)


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(), dict(dA=None, W=None), dict(dW=None, A=None),
                                dict(act=0, Z=None), dict(dA=None, dW=None, A=None, W=None)])
def test_linear_backward_accepts(kw):
    st, why = backward(**kw)
    assert st == tp.TPGEMM_ERR_ARCH, (st, why)


def norm(rows=6, cols=100, ldx=0, ldr=0, ldh=0, ldy=0, x=0, g=0, y=0, scale=0, eps=1e-5, Y=addr(0),
         H=addr(1), S=addr(2), rstd=addr(3), X=addr(4), R=addr(5), G=addr(6)):
    d = tp.RmsNormDesc(rows, cols, ldx, ldr, ldh, ldy, x, g, y, scale, eps)
    return tp.tpgemm_rmsnorm(Y, H, S, rstd, X, R, G, d, 0), tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(rows=-1), tp.TPGEMM_ERR_SHAPE, "rows=-1"),
    (dict(cols=0), tp.TPGEMM_ERR_SHAPE, "cols=0"),
    (dict(eps=-1.0), tp.TPGEMM_ERR_SHAPE, "eps"),
    (dict(eps=float("nan")), tp.TPGEMM_ERR_SHAPE, "eps"),
    (dict(ldx=99), tp.TPGEMM_ERR_SHAPE, "X: row stride 99"),
    (dict(x=tp.TPGEMM_ELEM_E4M3), tp.TPGEMM_ERR_DTYPE, "X must be"),
    (dict(g=tp.TPGEMM_ELEM_BF16), tp.TPGEMM_ERR_DTYPE, "gamma"),
    (dict(scale=3), tp.TPGEMM_ERR_DTYPE, "scale mode 3"),
    (dict(scale=1), tp.TPGEMM_ERR_DTYPE, "e4m3 or e5m2 with"),
    (dict(y=tp.TPGEMM_ELEM_E4M3), tp.TPGEMM_ERR_DTYPE, "without scales"),
    (dict(Y=None), tp.TPGEMM_ERR_NULL, "Y is NULL"),
    (dict(X=None), tp.TPGEMM_ERR_NULL, "X is NULL"),
    (dict(G=None), tp.TPGEMM_ERR_NULL, "gamma is NULL"),
    (dict(S=None, scale=2, y=3), tp.TPGEMM_ERR_NULL, "scale is NULL"),
    (dict(rstd=addr(3, 2)), tp.TPGEMM_ERR_ALIGN, "rstd="),
    (dict(Y=addr(4)), tp.TPGEMM_ERR_ALIAS, "Y overlaps X"),
    (dict(H=addr(5, 2)), tp.TPGEMM_ERR_ALIAS, "H overlaps R"),
    (dict(H=addr(4), ldh=108), tp.TPGEMM_ERR_ALIAS, "H overlaps X"),
    (dict(H=None, Y=addr(4), y=8), tp.TPGEMM_ERR_ALIAS, "Y overlaps X"),
    (dict(S=addr(0), scale=1, y=2), tp.TPGEMM_ERR_ALIAS, "Y overlaps scale"),
])
def test_rmsnorm_refuses(kw, status, frag):
    st, why = norm(**kw)
    assert st == status and frag in why, (st, why)


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(), dict(H=addr(4)), dict(H=addr(5)), dict(H=None, Y=addr(4)),
                                dict(R=None, rstd=None, S=None), dict(scale=1, y=2), dict(g=8)])
def test_rmsnorm_accepts(kw):
    st, why = norm(**kw)
    assert st == tp.TPGEMM_ERR_ARCH, (st, why)


def norm_grad(rows=6, cols=100, x=0, g=0, grad=8, dX=addr(0), dG=addr(1), dY=addr(2), H=addr(3),
              rstd=addr(4), G=addr(5), dH=addr(6), ws=addr(9), wsb=None, lddx=0):
    d = tp.RmsNormGradDesc(rows, cols, 0, 0, 0, lddx, x, g, grad)
    if wsb is None:
        wsb = tp.tpgemm_rmsnorm_backward_workspace_bytes(rows, cols)
    st = tp.tpgemm_rmsnorm_backward(dX, dG, dY, H, rstd, G, dH, d, ws, wsb, 0)
    return st, tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(cols=0), tp.TPGEMM_ERR_SHAPE, "cols=0"),
    (dict(x=2), tp.TPGEMM_ERR_DTYPE, "dY must be"),
    (dict(grad=2), tp.TPGEMM_ERR_DTYPE, "dgamma"),
    (dict(g=1), tp.TPGEMM_ERR_DTYPE, "gamma"),
    (dict(dY=None), tp.TPGEMM_ERR_NULL, "dY is NULL"),
    (dict(H=None), tp.TPGEMM_ERR_NULL, "H is NULL"),
    (dict(rstd=None), tp.TPGEMM_ERR_NULL, "rstd is NULL"),
    (dict(G=None), tp.TPGEMM_ERR_NULL, "gamma is NULL"),
    (dict(dX=addr(2), lddx=104), tp.TPGEMM_ERR_ALIAS, "dX overlaps dY"),
    (dict(dX=addr(3, 2)), tp.TPGEMM_ERR_ALIAS, "dX overlaps H"),
    (dict(dG=addr(0)), tp.TPGEMM_ERR_ALIAS, "dX overlaps dgamma"),
    (dict(ws=None), tp.TPGEMM_ERR_NULL, "workspace is NULL"),
    (dict(wsb=4), tp.TPGEMM_ERR_NULL, "workspace of 4 bytes"),
    (dict(ws=addr(6)), tp.TPGEMM_ERR_ALIAS, "workspace overlaps dH"),
])
def test_rmsnorm_backward_refuses(kw, status, frag):
    st, why = norm_grad(**kw)
    assert st == status and frag in why, (st, why)


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(), dict(dX=addr(2)), dict(dX=addr(3)), dict(dX=addr(6)),
                                dict(dH=None), dict(dG=None, ws=None), dict(dX=None, G=None)])
def test_rmsnorm_backward_accepts(kw):
    st, why = norm_grad(**kw)
    assert st == tp.TPGEMM_ERR_ARCH, (st, why)


def test_a_null_description_is_refused():
    lib = tp.library()
    assert lib.tpgemm_linear(*[None] * 8, None, None, 0, None) == tp.TPGEMM_ERR_NULL
    assert lib.tpgemm_linear_backward(*[None] * 7, None, None, 0, None) == tp.TPGEMM_ERR_NULL
    assert lib.tpgemm_rmsnorm(*[None] * 7, None, None) == tp.TPGEMM_ERR_NULL
    assert lib.tpgemm_rmsnorm_backward(*[None] * 7, None, None, 0, None) == tp.TPGEMM_ERR_NULL
    assert lib.tpgemm_linear_workspace_bytes(None, None, None) == 0
    assert lib.tpgemm_linear_backward_workspace_bytes(None, None, None, None) == 0


def test_the_python_forms_refuse_what_is_not_on_a_gpu():
    a = torch.zeros(4, 8, dtype=torch.float16)
    v = torch.ones(8, dtype=torch.float16)
    for call in (lambda: tp.linear(a, a), lambda: tp.linear_backward(a, a, a),
                 lambda: tp.rmsnorm(a, v), lambda: tp.rmsnorm_backward(a, a, v, v)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="2-D"):
        tp.linear(v, a)
