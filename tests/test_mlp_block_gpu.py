"""The example's feed-forward block, which chains the norm, the linear layer and their gradients,
against the same block in 64 bits (GPU only)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROUND = 2.0 ** -9  # of a bfloat16 store, relative


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tile_primitive_tensor_gb300 import build as tpbuild
    tpbuild.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "mlp_block.py")
    spec = importlib.util.spec_from_file_location("mlp_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


# Distances are of whole tensors. Each bfloat16 store on the way (h, y, u and out forward; the stored
# value before the activation, du, dz, dy and dx backward) moves its tensor by at most ROUND of its
# norm, which the norm, the activation and the products of random matrices pass on with a factor of
# at most 2. An e4m3 value is within 2^-4 of its own; two of them meet in each term of a product.
@pytest.mark.parametrize("tokens,width,hidden", [(1, 256, 512), (7, 264, 520), (16, 1024, 2048),
                                                 (100, 520, 264), (513, 512, 1536)])
def test_block(block, tokens, width, hidden):
    e = block.errors(tokens, width, hidden, seed=tokens)
    assert e.pop("out") <= 2 * 4 * ROUND
    assert e.pop("served") <= 2 * 2.0 ** -4 + 2 * 4 * ROUND
    for name, v in e.items():
        assert v <= 2 * 9 * ROUND, name
