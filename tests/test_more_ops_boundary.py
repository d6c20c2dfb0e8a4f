"""What the layer norm, dropout and the gated linear layer refuse, without a GPU: every rejection
names its reason before anything is enqueued. Pointers are fake addresses that these paths never
read. And the known answers of the random words' generator that the tests compare with."""
import numpy as np
import pytest
import torch

import more_ops_reference as more
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


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake addresses")


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_words(counter, key, words):
    got = more.philox(*[np.array([c], dtype=np.uint64) for c in counter], *key)
    assert tuple(int(w[0]) for w in got) == words


def dropout(rows=6, cols=100, ldx=0, ldr=0, ldy=0, x=0, p=0.1, counter=None, Y=addr(0), X=addr(1), R=addr(2)):
    d = tp.DropoutDesc(rows, cols, ldx, ldr, ldy, x, p, 1, 2, counter)
    return tp.tpgemm_dropout(Y, X, R, d, 0), tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(rows=-1), tp.TPGEMM_ERR_SHAPE, "rows=-1"),
    (dict(cols=1 << 30), tp.TPGEMM_ERR_SHAPE, "cols=1073741824"),
    (dict(ldx=99), tp.TPGEMM_ERR_SHAPE, "X: row stride 99"),
    (dict(x=tp.TPGEMM_ELEM_E4M3), tp.TPGEMM_ERR_DTYPE, "X must be"),
    (dict(p=1.0), tp.TPGEMM_ERR_SHAPE, "p=1"),
    (dict(p=-0.5), tp.TPGEMM_ERR_SHAPE, "p=-0.5"),
    (dict(p=float("nan")), tp.TPGEMM_ERR_SHAPE, "p="),
    (dict(counter=addr(3, 4)), tp.TPGEMM_ERR_ALIGN, "counter="),
    (dict(counter=addr(0, 8)), tp.TPGEMM_ERR_ALIAS, "Y overlaps counter"),
    (dict(X=None), tp.TPGEMM_ERR_NULL, "X is NULL"),
    (dict(Y=None), tp.TPGEMM_ERR_NULL, "Y is NULL"),
    (dict(Y=addr(0, 1)), tp.TPGEMM_ERR_ALIGN, "Y="),
    (dict(Y=addr(1, 2)), tp.TPGEMM_ERR_ALIAS, "Y overlaps X"),
    (dict(Y=addr(2), ldy=104), tp.TPGEMM_ERR_ALIAS, "Y overlaps R"),
])
def test_dropout_refuses(kw, status, frag):
    st, why = dropout(**kw)
    assert st == status and frag in why, (st, why)


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(), dict(Y=addr(1)), dict(Y=addr(2)), dict(R=None), dict(counter=addr(3, 8)),
                                dict(p=0.0, counter=addr(0, 8))])
def test_dropout_accepts(kw):
    st, why = dropout(**kw)
    assert st == tp.TPGEMM_ERR_ARCH, (st, why)


def norm(rows=6, cols=100, ldx=0, ldr=0, ldh=0, ldy=0, x=0, g=0, y=0, scale=0, eps=1e-5, p=0.0, counter=None,
         Y=addr(0), H=addr(1), S=addr(2), mean=addr(3), rstd=addr(4), X=addr(5), R=addr(6), G=addr(7), B=addr(8)):
    d = tp.LayerNormDesc(rows, cols, ldx, ldr, ldh, ldy, x, g, y, scale, eps, p, 1, 2, counter)
    return tp.tpgemm_layernorm(Y, H, S, mean, rstd, X, R, G, B, d, 0), tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(rows=-1), tp.TPGEMM_ERR_SHAPE, "rows=-1"),
    (dict(cols=0), tp.TPGEMM_ERR_SHAPE, "cols=0"),
    (dict(eps=-1.0), tp.TPGEMM_ERR_SHAPE, "eps"),
    (dict(eps=float("nan")), tp.TPGEMM_ERR_SHAPE, "eps"),
    (dict(p=1.5), tp.TPGEMM_ERR_SHAPE, "p=1.5"),
    (dict(ldh=99), tp.TPGEMM_ERR_SHAPE, "H: row stride 99"),
    (dict(x=tp.TPGEMM_ELEM_E5M2), tp.TPGEMM_ERR_DTYPE, "X must be"),
    (dict(g=tp.TPGEMM_ELEM_BF16), tp.TPGEMM_ERR_DTYPE, "gamma and beta"),
    (dict(scale=tp.TPGEMM_SCALE_MX, y=tp.TPGEMM_ELEM_E4M3), tp.TPGEMM_ERR_DTYPE, "scale mode 2"),
    (dict(scale=1), tp.TPGEMM_ERR_DTYPE, "Y must be"),
    (dict(y=tp.TPGEMM_ELEM_E4M3), tp.TPGEMM_ERR_DTYPE, "Y must be"),
    (dict(scale=1, y=tp.TPGEMM_ELEM_E4M3, S=None), tp.TPGEMM_ERR_NULL, "scale is NULL"),
    (dict(X=None), tp.TPGEMM_ERR_NULL, "X is NULL"),
    (dict(G=None), tp.TPGEMM_ERR_NULL, "gamma is NULL"),
    (dict(mean=addr(3, 2)), tp.TPGEMM_ERR_ALIGN, "mean="),
    (dict(Y=addr(5)), tp.TPGEMM_ERR_ALIAS, "Y overlaps X"),
    (dict(Y=addr(1, 16)), tp.TPGEMM_ERR_ALIAS, "Y overlaps H"),
    (dict(mean=addr(4, 8)), tp.TPGEMM_ERR_ALIAS, "mean overlaps rstd"),
    (dict(rstd=addr(8, 4)), tp.TPGEMM_ERR_ALIAS, "rstd overlaps beta"),
    (dict(p=0.1, counter=addr(1, 8)), tp.TPGEMM_ERR_ALIAS, "H overlaps counter"),
])
def test_layernorm_refuses(kw, status, frag):
    st, why = norm(**kw)
    assert st == status and frag in why, (st, why)


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(), dict(H=addr(5)), dict(H=addr(6)), dict(H=None, Y=addr(6)),
                                dict(H=None, R=None, B=None, mean=None, rstd=None, S=None),
                                dict(scale=1, y=tp.TPGEMM_ELEM_E5M2), dict(p=0.5, counter=addr(9))])
def test_layernorm_accepts(kw):
    st, why = norm(**kw)
    assert st == tp.TPGEMM_ERR_ARCH, (st, why)


def norm_backward(rows=6, cols=100, x=0, g=0, grad=8, p=0.0, dX=addr(0), dR=addr(1), dG=addr(2), dB=addr(3),
                  dY=addr(4), H=addr(5), mean=addr(6), rstd=addr(7), G=addr(8), dH=addr(9), ws=addr(10), wsb=None,
                  **lds):
    d = tp.LayerNormGradDesc(rows, cols, *[lds.get(n, 0) for n in ("lddy", "ldh", "lddh", "lddx", "lddr")], x, g,
                             grad, p, 1, 2, None)
    if wsb is None:
        wsb = tp.tpgemm_layernorm_backward_workspace_bytes(rows, cols)
    st = tp.tpgemm_layernorm_backward(dX, dR, dG, dB, dY, H, mean, rstd, G, dH, d, ws, wsb, 0)
    return st, tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(rows=-1), tp.TPGEMM_ERR_SHAPE, "rows=-1"),
    (dict(grad=tp.TPGEMM_ELEM_E5M2), tp.TPGEMM_ERR_DTYPE, "dgamma and dbeta"),
    (dict(p=1.0), tp.TPGEMM_ERR_SHAPE, "p=1"),
    (dict(dY=None), tp.TPGEMM_ERR_NULL, "dY is NULL"),
    (dict(mean=None), tp.TPGEMM_ERR_NULL, "mean is NULL"),
    (dict(G=None), tp.TPGEMM_ERR_NULL, "gamma is NULL"),
    (dict(lddr=99), tp.TPGEMM_ERR_SHAPE, "dR: row stride 99"),
    (dict(dX=addr(1)), tp.TPGEMM_ERR_ALIAS, "dX overlaps dR"),
    (dict(dR=addr(5, 2)), tp.TPGEMM_ERR_ALIAS, "dR overlaps H"),
    (dict(dB=addr(8)), tp.TPGEMM_ERR_ALIAS, "dbeta overlaps gamma"),
    (dict(ws=None), tp.TPGEMM_ERR_NULL, "workspace is NULL"),
    (dict(ws=addr(10, 64)), tp.TPGEMM_ERR_ALIGN, "256-byte"),
    (dict(wsb=256), tp.TPGEMM_ERR_NULL, "workspace of 256 bytes"),
    (dict(ws=addr(4)), tp.TPGEMM_ERR_ALIAS, "workspace overlaps dY"),
])
def test_layernorm_backward_refuses(kw, status, frag):
    st, why = norm_backward(**kw)
    assert st == status and frag in why, (st, why)


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(), dict(dX=addr(4)), dict(dX=addr(5), dR=addr(9)), dict(dX=addr(9)),
                                dict(dG=None, dB=None, ws=None), dict(dX=None, dR=None, G=None, dG=None),
                                dict(p=0.5, dH=None)])
def test_layernorm_backward_accepts(kw):
    st, why = norm_backward(**kw)
    assert st == tp.TPGEMM_ERR_ARCH, (st, why)


def gated(M=24, N=40, K=64, lda=0, ldw=0, ldy=0, ldz=0, dtype=tp.TPGEMM_ELEM_F16, out=tp.TPGEMM_ELEM_F16, act=2,
          Y=addr(0), Z=addr(1), A=addr(2), W=addr(3), sa=None, sw=None, bias=addr(4), ws=None, wsb=0):
    d = tp.LinearDesc(M, N, K, lda, ldw, 0, ldy, ldz, dtype, out, act)
    st = tp.tpgemm_gated_linear(Y, Z, A, W, sa, sw, bias, d, ws, wsb, 0)
    return st, tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(M=-1), tp.TPGEMM_ERR_SHAPE, "M=-1"),
    (dict(N=1 << 29), tp.TPGEMM_ERR_SHAPE, "2 N=1073741824"),
    (dict(ldw=63), tp.TPGEMM_ERR_SHAPE, "W: row stride 63"),
    (dict(ldz=79), tp.TPGEMM_ERR_SHAPE, "Z: row stride 79"),
    (dict(dtype=tp.TPGEMM_ELEM_F32), tp.TPGEMM_ERR_DTYPE, "dtype 8"),
    (dict(out=tp.TPGEMM_ELEM_E4M3), tp.TPGEMM_ERR_DTYPE, "out 2"),
    (dict(act=5), tp.TPGEMM_ERR_DTYPE, "activation 5"),
    (dict(sw=addr(6)), tp.TPGEMM_ERR_DTYPE, "e4m3 or e5m2"),
    (dict(Y=None), tp.TPGEMM_ERR_NULL, "Y is NULL"),
    (dict(W=None), tp.TPGEMM_ERR_NULL, "W is NULL"),
    (dict(bias=addr(4, 1)), tp.TPGEMM_ERR_ALIGN, "bias="),
    # the second half of what has 2 N rows or columns counts
    (dict(Y=addr(3, 2 * 79 * 64)), tp.TPGEMM_ERR_ALIAS, "Y overlaps W"),
    (dict(Z=addr(0, -2 * (24 * 80 - 1))), tp.TPGEMM_ERR_ALIAS, "Y overlaps Z"),
    (dict(Y=addr(4, 2 * 79)), tp.TPGEMM_ERR_ALIAS, "Y overlaps bias"),
    (dict(A=addr(2, 2)), tp.TPGEMM_ERR_NULL, "workspace is NULL"),
])
def test_gated_linear_refuses(kw, status, frag):
    st, why = gated(**kw)
    assert st == status and frag in why, (st, why)


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(), dict(Z=None, bias=None), dict(K=0, A=None, W=None), dict(A=addr(2, 2)),
                                dict(dtype=tp.TPGEMM_ELEM_E5M2, sa=addr(6), sw=addr(7), out=8)])
def test_gated_linear_accepts(kw):
    need = tp.tpgemm_gated_linear_workspace_bytes(
        kw.get("A", addr(2)), addr(3), tp.LinearDesc(24, 40, kw.get("K", 64), 0, 0, 0, 0, 0, kw.get("dtype", 0), 0, 0))
    st, why = gated(**kw, ws=addr(9) if need else None, wsb=need)
    assert st == tp.TPGEMM_ERR_ARCH, (st, why)


def gated_backward(M=24, N=40, K=64, dtype=0, grad=8, act=2, dA=addr(0), dW=addr(1), db=addr(2), dY=addr(3),
                   A=addr(4), W=addr(5), Z=addr(6), ws=addr(9), wsb=None, **lds):
    d = tp.LinearGradDesc(M, N, K, *[lds.get(n, 0) for n in ("lddy", "ldz", "lda", "ldw", "ldda", "lddw")],
                          dtype, grad, act)
    if wsb is None:
        wsb = tp.tpgemm_gated_linear_backward_workspace_bytes(dY, A, W, d)
    st = tp.tpgemm_gated_linear_backward(dA, dW, db, dY, A, W, Z, d, ws, wsb, 0)
    return st, tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(N=1 << 29), tp.TPGEMM_ERR_SHAPE, "2 N="),
    (dict(dtype=tp.TPGEMM_ELEM_E4M3), tp.TPGEMM_ERR_DTYPE, "f16 or bf16"),
    (dict(Z=None), tp.TPGEMM_ERR_NULL, "Z is NULL"),
    (dict(Z=None, act=0), tp.TPGEMM_ERR_NULL, "Z is NULL"),
    (dict(ldz=79), tp.TPGEMM_ERR_SHAPE, "Z: row stride 79"),
    (dict(dW=addr(5, 2 * 64 * 80 - 2)), tp.TPGEMM_ERR_ALIGN, "dW="),
    (dict(dW=addr(5, 2 * 64 * 80 - 4)), tp.TPGEMM_ERR_ALIAS, "dW overlaps W"),
    (dict(db=addr(1, 4 * 64 * 80 - 4)), tp.TPGEMM_ERR_ALIAS, "dW overlaps dbias"),
    (dict(ws=None), tp.TPGEMM_ERR_NULL, "workspace is NULL"),
    (dict(wsb=512), tp.TPGEMM_ERR_NULL, "workspace of 512 bytes"),
    (dict(ws=addr(6)), tp.TPGEMM_ERR_ALIAS, "workspace overlaps Z"),
])
def test_gated_linear_backward_refuses(kw, status, frag):
    st, why = gated_backward(**kw)
    assert st == status and frag in why, (st, why)


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(), dict(act=0), dict(dA=None, W=None), dict(dW=None, A=None)])
def test_gated_linear_backward_accepts(kw):
    st, why = gated_backward(**kw)
    assert st == tp.TPGEMM_ERR_ARCH, (st, why)


def test_python_refuses_before_the_library():
    a = torch.zeros(4, 8)
    for call in (lambda: tp.gated_linear(a, torch.zeros(6, 8)), lambda: tp.layernorm(a, torch.zeros(8)),
                 lambda: tp.dropout(a, tp.Dropout(0.1, 1))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
