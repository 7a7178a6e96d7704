"""Scales that 32-bit floats cannot hold are refused on the host: as 0 or infinity in a kernel, a hidden key's -inf times such a
scale would be NaN. Fake pointers are never touched: every case fails validation first."""
import pytest

from test_abi_network_cpu import L, _attn, _loss  # noqa: F401  (L is a fixture)


@pytest.mark.parametrize("scale", [1e-46, 1e-40, 5e38, 1e300, 2.5e38])      # the last: times log2(e) beyond the largest float
@pytest.mark.parametrize("backward", [False, True])
def test_attention_scale(L, scale, backward):  # noqa: F811
    assert _attn(L, backward=backward, scale=scale) == -1


@pytest.mark.parametrize("t", [1e-46, 1e-39, 2.5e38 ** -1, 1e39, 1e300, 1.7e38])      # 1 / 1.7e38 is below the normal range
@pytest.mark.parametrize("backward", [False, True])
def test_matching_loss_temperature(L, t, backward):  # noqa: F811
    assert _loss(L, backward=backward, t=t) == -1
