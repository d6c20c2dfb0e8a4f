"""Outputs that are slices of wider rows: what lies between a row's end and the next one's start, and
behind the last row, stays as it was (GPU only). Strides are multiples of 16 bytes, widths are not:
a store of whole 16-byte units writes more than the row."""
import pytest
import torch

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


class Slice:
    """A [rows, cols] view of rows of `ld` values that are all 7, with some behind the last."""

    def __init__(self, rows, cols, dtype, ld):
        self.buf = torch.full((rows * ld + 64,), 7.0, dtype=dtype, device="cuda")
        self.view = self.buf.as_strided((rows, cols), (ld, 1))

    def surroundings_stay(self):
        mask = torch.ones(self.buf.numel(), dtype=torch.bool, device="cuda")
        mask.as_strided(self.view.shape, self.view.stride()).fill_(False)
        return bool((self.buf[mask] == 7).all())


def normal(*shape, dtype=BF16, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def up(n):
    return (n + 7) // 8 * 8


@pytest.mark.parametrize("path", ["tile", "split", "few"])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("M", [1, 13, 300])
def test_linear_layers(M, out, path, tune):
    if path == "few" and M > 16:
        pytest.skip("up to 16 tokens")
    tune.setenv("TPGEMM_LINEAR_PATH", path)
    K = 72
    A = normal(M, K)
    for N in (1, 3, 31, 33, 61, 62, 63, 65, 250, 255, 300):
        W = normal(2 * N, K, std=K ** -0.5)
        for kept in (False, True):
            y, z = Slice(M, N, out, up(N) + 8), Slice(M, N, out, up(N))
            r = normal(M, up(N), dtype=out)[:, :N]
            tp.linear(A, W[:N], None, None if kept else r, act="silu", out_dtype=out, out=y.view,
                      pre=z.view if kept else None)
            assert y.surroundings_stay() and z.surroundings_stay(), ("linear", N, kept)
            want, _, bound, _ = ref.linear(A, W[:N], None, None if kept else r, "silu", None, None, out)
            ok, why = ref.within(y.view, want, bound)
            assert ok, ("linear", N, kept, why)
            y, z = Slice(M, N, out, up(N)), Slice(M, 2 * N, out, up(2 * N))
            tp.gated_linear(A, W, out_dtype=out, out=y.view, pre=z.view if kept else None)
            assert y.surroundings_stay() and (not kept or z.surroundings_stay()), ("gated", N, kept)


@pytest.mark.parametrize("path", ["tile", "split"])
@pytest.mark.parametrize("K", [1, 33, 62, 255])
def test_gradients(K, path, tune):
    # (through the C entry: the Python calls make dense outputs)
    tune.setenv("TPGEMM_LINEAR_PATH", path)
    M, N = 300, 72
    A, W, dY, pre = normal(M, K), normal(2 * N, K), normal(M, N), normal(M, 2 * N)
    for gated in (False, True):
        rows = 2 * N if gated else N
        for grad, code in ((BF16, tp.TPGEMM_ELEM_BF16), (F32, tp.TPGEMM_ELEM_F32)):
            dA, dW, db = Slice(M, K, BF16, up(K)), Slice(rows, K, grad, up(K)), Slice(1, rows, grad, rows)
            d = tp.LinearGradDesc(M, N, K, 0, 0, 0, 0, up(K), up(K), tp.TPGEMM_ELEM_BF16, code, tp.TPGEMM_ACT_SILU)
            size, call = ((tp.tpgemm_gated_linear_backward_workspace_bytes, tp.tpgemm_gated_linear_backward) if gated else
                          (tp.tpgemm_linear_backward_workspace_bytes, tp.tpgemm_linear_backward))
            need = size(dY, A, W, d)
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
            assert call(dA.view, dW.view, db.view, dY, A, W[:rows], pre, d, ws, need,
                        torch.cuda.current_stream()) == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()
            torch.cuda.synchronize()
            assert dA.surroundings_stay() and dW.surroundings_stay() and db.surroundings_stay(), (gated, grad)
            z = pre if gated else pre.view(-1)[:M * N].view(M, N)
            call = tp.gated_linear_backward if gated else tp.linear_backward
            want = call(dY, A, W[:rows], z, act="silu", grad_dtype=grad)
            for got, w in zip((dA.view, dW.view), want):
                assert float((got.double() - w.double()).norm()) <= 2.0 ** -6 * float(w.double().norm())
