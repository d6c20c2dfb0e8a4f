"""Limits of the operators around the multiply that need no GPU: strides at the end of 64 bits, and
when the linear layer asks for a workspace. Pointers are fake addresses that these paths never read."""
import pytest

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


def linear(M=8, N=8, K=8, lda=0, ldw=0, ldr=0, ldy=0, ldz=0, dtype=tp.TPGEMM_ELEM_F16):
    d = tp.LinearDesc(M, N, K, lda, ldw, ldr, ldy, ldz, dtype, tp.TPGEMM_ELEM_F16, 0)
    st = tp.tpgemm_linear(addr(0), addr(1), addr(2), addr(3), None, None, addr(4), addr(5), d, None, 0, 0)
    return st, tp.tpgemm_last_error_detail()


@pytest.mark.parametrize("kw,name", [
    (dict(M=1 << 29, lda=1 << 38), "A"),  # 2^29 (2^35 + 1) 16-byte units: 2^29 of them, cut off at 64 bits
    (dict(M=(1 << 30) - 1, ldy=1 << 40), "Y"),
    (dict(M=1 << 26, ldr=1 << 40), "R"),
    (dict(N=1 << 26, ldw=1 << 40), "W"),
])
def test_strides_whose_span_wraps_around_are_refused(kw, name):
    st, why = linear(**kw)
    assert st == tp.TPGEMM_ERR_SHAPE and why.startswith(f"{name} exceeds"), (st, why)


# linear in Python asks for the workspace's size only where an operand's rows are off the 128-byte
# lines: on them none is needed, whatever the sizes, types and kernel.
@pytest.mark.parametrize("dtype,size", [(tp.TPGEMM_ELEM_BF16, 2), (tp.TPGEMM_ELEM_E4M3, 1)])
@pytest.mark.parametrize("path", [None, "tile", "split", "few"])
def test_operands_on_whole_lines_need_no_workspace(dtype, size, path, tune):
    if path:
        tune.setenv("TPGEMM_LINEAR_PATH", path)
    line = 128 // size
    for M in (1, 16, 17, 48, 144, 257, 4096):
        for N in (1, 1000, 16384):
            for K in (1, line - 1, 1000, 16384):
                ld = -(-K // line) * line
                for lda, ldw in ((ld, ld), (ld + line, ld), (ld, 3 * ld)):
                    d = tp.LinearDesc(M, N, K, lda, ldw, 0, 0, 0, dtype, tp.TPGEMM_ELEM_F16, 0)
                    assert tp.tpgemm_linear_workspace_bytes(addr(2), addr(3), d) == 0


def test_operands_off_the_lines_may_need_one():
    def need(M, N, K, A, W):
        return tp.tpgemm_linear_workspace_bytes(A, W, tp.LinearDesc(M, N, K, 0, 0, 0, 0, 0, tp.TPGEMM_ELEM_F16, 0, 0))
    assert need(40, 40, 1001, addr(2), addr(3)) > 0  # rows off 16 bytes
    assert need(40, 40, 1024, addr(2, 2), addr(3)) > 0  # a start off 16 bytes
    assert need(144, 16384, 4104, addr(2), addr(3)) > 0  # few tokens off the lines, large weights
    assert need(16, 40, 1001, addr(2), addr(3)) == 0  # up to 16 tokens are read as they lie
