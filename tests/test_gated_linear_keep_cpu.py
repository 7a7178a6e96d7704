"""The differentiable gated layer keeps its projections only where a gradient may be asked for. The kernels' call is replaced by one
that notes what it is asked to keep, so no GPU is needed."""
import pytest
import torch

import dense_descriptor_matching_amd as ddm


@pytest.fixture
def asked(monkeypatch):
    """What calls asked to keep, in their order."""
    seen = []

    def forward(x, weight, bias=None, *, activation="silu", keep=False):
        seen.append(keep)
        hidden = weight.shape[0] // 2
        return x.new_zeros(x.shape[:-1] + (hidden,)), x.new_zeros(x.shape[:-1] + (2 * hidden,)) if keep else None

    monkeypatch.setattr(ddm.network, "gated_linear_forward", forward)
    return seen


def tensors(*needs):
    return [t.requires_grad_(n) for t, n in zip((torch.ones(3, 4), torch.ones(10, 4), torch.ones(10)), needs)]


@pytest.mark.parametrize("needs", [(True, True, True), (False, True, True), (False, False, True), (True, False, False)])
def test_kept_for_a_gradient_alone(asked, needs):
    t = tensors(*needs)
    assert ddm.gated_linear(*t).requires_grad
    with torch.no_grad():
        assert not ddm.gated_linear(*t).requires_grad
        with torch.enable_grad():
            assert ddm.gated_linear(*t).requires_grad
    with torch.inference_mode():
        ddm.gated_linear(*t)
    assert asked == [True, False, True, False]


def test_nothing_to_keep_without_leaves(asked):
    assert not ddm.gated_linear(*tensors(False, False, False)).requires_grad
    ddm.gated_linear(*tensors(False, False, False)[:2])
    assert asked == [False, False]
