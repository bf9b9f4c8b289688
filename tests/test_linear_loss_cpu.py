"""What the autograd form of the linear cross entropy refuses, without a GPU."""
import pytest
import torch

import mixed_precision_optimizer_mta_amd as M


def test_weights_that_want_a_gradient():
    """There is none for them: refused, not left at None, unless nobody asks."""
    h, w = torch.zeros(4, 8), torch.zeros(5, 8)
    t = torch.zeros(4, dtype=torch.int64)
    wt = torch.ones(4, requires_grad=True)
    for weights in (wt, wt * 2):
        with pytest.raises(ValueError, match="no gradient for weights"):
            M.linear_cross_entropy(h, w, t, weights=weights)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            M.linear_cross_entropy(h, w, t, weights=weights)
        with pytest.raises(ValueError, match="GPU"):
            M.linear_cross_entropy(h, w, t, weights=weights.detach())
