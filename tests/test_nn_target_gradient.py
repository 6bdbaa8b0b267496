"""distill_loss has no gradient to the teacher's values; a caller that asks for
one is told so."""
import pytest
import torch

from float8_mixed_precision_gb300 import nn as f8nn


def test_values_with_a_gradient_are_refused():
    z = torch.zeros((2, 40), requires_grad=True)
    ids, values = torch.zeros((2, 4), dtype=torch.int32), torch.zeros((2, 4), requires_grad=True)
    with pytest.raises(ValueError, match="values"):
        f8nn.distill_loss(z, ids, values)
    # without a gradient to form there is nothing to lose; host tensors are refused next
    with torch.no_grad(), pytest.raises(ValueError, match="device tensors"):
        f8nn.distill_loss(z, ids, values)
    with pytest.raises(ValueError, match="device tensors"):
        f8nn.distill_loss(z, ids, values.detach())
