"""An output that nothing would be written to is refused, without a GPU."""
import pytest
import torch

import tile_primitive_tensor_gb300 as tp


@pytest.mark.parametrize("need,drop", [((False, True, True, True), True), ((False, False, True, True), True),
                                       ((False, False, True, True), False)])
def test_layernorm_backward_refuses_an_output_that_it_would_not_write(need, drop):
    a, v = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="out"):
        tp.layernorm_backward(a, a, v[:4], v[:4], v, dropout=tp.Dropout(0.1, 1) if drop else None, need=need,
                              out=torch.zeros(4, 8))
