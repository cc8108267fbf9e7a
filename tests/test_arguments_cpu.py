"""Arguments that the Python wrappers refuse before they look at a tensor.  No call reaches a GPU."""
import pytest
import torch

import bit_nf4_quantized_19_b200 as q


@pytest.mark.parametrize("given", [(), ("dA",), ("dB",)])
def test_accumulate_needs_both_gradients(given):
    """Without both there is nothing to add into: linear_bwd made them up from unwritten memory."""
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    g = {k: torch.zeros(128, 128) for k in given}
    with pytest.raises(ValueError):
        q.linear_bwd(x, x, None, None, x, x, 1.0, accumulate=True, **g)
