"""The layer norm, dropout and the gated linear layer on a given stream while the current one is busy
(GPU only): as the other operators, an output is never memory that work on the current stream still
reads, and a dropped one does not come back while its stream writes. Two calls at once on two
streams, and rows that lie more than 2^32 bytes apart."""
import pytest
import torch

import more_ops_reference as more
import ops_reference as ref
import test_ops_streams_gpu as streams
import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

N = streams.N


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    yield
    assert tp.tpgemm_last_device_error() == tp.TPGEMM_OK, tp.tpgemm_last_error_detail()


def calls():
    """Name, and a call whose largest outputs are [N, N] of 16 bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.randn(N, N, generator=g, device="cuda").half() for _ in range(2))
    wide = torch.randn(2 * N, N, generator=g, device="cuda").half()
    pre = torch.randn(N, 2 * N, generator=g, device="cuda").half()
    w, rstd = torch.ones(N, device="cuda").half(), torch.ones(N, device="cuda")
    d = tp.Dropout(0.1, 1, 2)
    return {"gated_linear": lambda s: tp.gated_linear(a, wide, stream=s),
            "gated_linear_backward": lambda s: tp.gated_linear_backward(b, a, wide, pre, stream=s)[0],
            "layernorm": lambda s: tp.layernorm(a, w, w, b, dropout=d, need_stats=True, stream=s).h,
            "layernorm_backward": lambda s: tp.layernorm_backward(a, b, rstd, rstd, w, b, dropout=d,
                                                                  stream=s).dresidual,
            "dropout": lambda s: tp.dropout(a, d, b, stream=s),
            "dropout_backward": lambda s: tp.dropout_backward(a, d, stream=s)}


NAMES = ["gated_linear", "gated_linear_backward", "layernorm", "layernorm_backward", "dropout",
         "dropout_backward"]


@pytest.mark.parametrize("kind", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_taken_from_the_current_stream(name, kind, monkeypatch):
    monkeypatch.setattr(streams, "calls", calls)
    streams.test_outputs_are_not_taken_from_the_current_stream(name, kind)


@pytest.mark.parametrize("name", NAMES)
def test_dropped_outputs_do_not_come_back_to_the_current_stream(name, monkeypatch):
    monkeypatch.setattr(streams, "calls", calls)
    streams.test_dropped_outputs_do_not_come_back_to_the_current_stream(name)


@pytest.mark.parametrize("name", NAMES)
def test_two_calls_at_once(name):
    call = calls()[name]
    want = call(None).clone()
    torch.cuda.synchronize()
    pair = [torch.cuda.Stream() for _ in range(2)]
    got = [call(pair[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("cols", [200, 201])
def test_rows_far_apart(cols):
    # 3 rows, 2^31 + 8 elements from one to the next: 12.9 GB
    ld = 2 ** 31 + 8
    flat = torch.empty(2 * ld + cols, dtype=torch.float16, device="cuda")
    x = flat.as_strided((3, cols), (ld, 1))
    near = torch.randn(3, cols, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    x.copy_(near)
    d = tp.Dropout(0.25, 3, 4)
    w, b = near[0].clone(), near[1].clone()
    assert torch.equal(tp.dropout(x, d), tp.dropout(near, d))
    for a, c in zip(tp.layernorm(x, w, b, x, dropout=d, need_stats=True),
                    tp.layernorm(near, w, b, near, dropout=d, need_stats=True)):
        assert (a is None and c is None) or torch.equal(a, c)
    mean, rstd = torch.zeros(3, device="cuda"), torch.ones(3, device="cuda")
    for a, c in zip(tp.layernorm_backward(x, x, mean, rstd, w, x, dropout=d),
                    tp.layernorm_backward(near, near, mean, rstd, w, near, dropout=d)):
        assert torch.equal(a, c)
    W = torch.randn(32, cols, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").half()
    assert torch.equal(tp.gated_linear(x, W), tp.gated_linear(near, W))
    assert torch.equal(tp.dropout(near, d, out=x), tp.dropout(near, d))


def test_more_than_2_to_32_elements():
    # 70000 x 65536 of 16 bits, 9.2 GB: rows at the end against the mask drawn on the host
    rows, cols = 70000, 65536
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    y = tp.dropout(x, tp.Dropout(0.5, 11, 12), out=x)
    n = -(-cols // 4)
    import numpy as np
    for row in (0, 65535, 65536, rows - 1):
        b = np.arange(n, dtype=np.uint64)
        w = np.stack(more.philox(b, np.full_like(b, row), np.full_like(b, 12), np.zeros_like(b), 11, 0), -1)
        keep = torch.from_numpy(w.reshape(-1)[:cols] >= np.uint64(2 ** 31)).cuda()
        assert torch.equal(y[row].float(), keep.float() * 2)


@pytest.mark.parametrize("name", ["layernorm", "dropout"])
def test_many_short_rows(name):
    # more rows than 2^20, in whole pieces and not
    for cols in (8, 5):
        x = torch.randn(1_100_000, cols, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
        if name == "dropout":
            y, err = more.drop(x, (0.5, 1, 2))
            got = tp.dropout(x, tp.Dropout(0.5, 1, 2))
        else:
            w, b = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
            (y, _, _, _), (err, _, _, _) = more.layernorm(x, w, b, None, 1e-5)
            got = tp.layernorm(x, w, b).y
        ok, why = ref.within(got, y, more.rounded(err, y, torch.float32))
        assert ok, why
