"""Rotary positions are differentiable by queries and keys. Frequencies or a magnitude that require a gradient are refused, before
anything else is looked at: they would get none."""
import pytest
import torch

import dense_descriptor_matching_amd as ddm


@pytest.mark.parametrize("k", [False, True])
def test_learned_frequencies_are_refused(k):
    q, pos, f = torch.ones(3, 2, 8), torch.arange(3, dtype=torch.int32), ddm.rotary_frequencies(4)
    k = torch.ones(3, 1, 8) if k else None
    with pytest.raises(ValueError, match="gradient"):
        ddm.rotary(q, k, pos, f.clone().requires_grad_())
    with pytest.raises(ValueError, match="gradient"):
        ddm.rotary(q, k, pos, f, magnitude=torch.tensor(1.5, requires_grad=True))
    learned = f.clone().requires_grad_()
    with torch.no_grad(), pytest.raises(TypeError, match="device tensor"):      # no gradient is asked for: the next check speaks
        ddm.rotary(q, k, pos, learned)
    with pytest.raises(TypeError, match="device tensor"):
        ddm.rotary(q, k, pos, learned.detach())
