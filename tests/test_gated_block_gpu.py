"""The example's gated block, which chains the layer norm, dropout, the gated and the plain linear layer
and their gradients, against the same block in 64 bits; and the chain captured into a graph that
draws new masks (GPU only)."""
import importlib.util
import os

import pytest
import torch

import tile_primitive_tensor_gb300 as tp

pytestmark = pytest.mark.gpu

ROUND = 2.0 ** -9  # of a bfloat16 store, relative


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "gated_block.py")
    spec = importlib.util.spec_from_file_location("gated_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


# Distances are of whole tensors. Each bfloat16 store on the way (h, n, [G | U], u, W2 u and y forward;
# the masked dy, du, dz, dn, dx and dr backward) moves its tensor by at most ROUND of its norm, which
# the norm, the gate and the products of random matrices pass on with a factor of at most 2 (a
# product of two rounded factors: of at most 3). An e4m3 value is within 2^-4 of its own; two of
# them meet in each term of G and of U, and both in u.
@pytest.mark.parametrize("tokens,width,hidden", [(1, 256, 512), (7, 264, 520), (16, 1024, 2048),
                                                 (100, 520, 264), (513, 512, 1536)])
@pytest.mark.parametrize("p_drop", [0.1, 0.5])
def test_block(block, tokens, width, hidden, p_drop):
    e = block.errors(tokens, width, hidden, seed=tokens, p_drop=p_drop)
    assert e.pop("out") <= 3 * 6 * ROUND
    assert e.pop("served") <= 2 * 2 * 2.0 ** -4 + 3 * 6 * ROUND
    for name, v in e.items():
        assert v <= 3 * 12 * ROUND, name


def test_captured_step_draws_anew(block):
    p = block.make_params(264, 520)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, dy = [torch.randn(40, 264, generator=g, device="cuda").bfloat16() for _ in range(3)]
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run(offset):
        drops = [tp.Dropout(0.2, 1, offset), tp.Dropout(0.2, 2, offset)]
        y, saved = block.forward(p, x, r, drops)
        return {"y": y, **block.backward(p, saved, dy, drops)}
    run(step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(step)
        step.add_(1)
    seen = []
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = run(i)
        for name, t in out.items():
            assert torch.equal(t, want[name]), name
        seen.append(out["y"].clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
