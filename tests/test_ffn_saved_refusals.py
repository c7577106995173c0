"""The gated block's backward pass refuses a forward pass that kept nothing:
``gated_product`` gives None for both without a checkpoint."""
import pytest
import torch

from combine_route_mask_amd import ffn as F, moe_ep as m

BF = torch.bfloat16


@pytest.mark.parametrize("missing", ["pre", "pre_scales", "both"])
def test_nothing_saved_is_refused(missing):
    x, w1, w2 = torch.zeros(2, 32, dtype=BF), torch.zeros(64, 32, dtype=BF), torch.zeros(32, 32, dtype=BF)
    pre, scales = torch.zeros(2, 64, dtype=torch.float16), torch.zeros(2, 8, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    pre, scales = None if missing in ("pre", "both") else pre, None if missing in ("pre_scales", "both") else scales
    with pytest.raises(m.MoeEpArgError, match="without one it keeps none"):
        F.gated_product_backward(x, w2, pre, scales)
