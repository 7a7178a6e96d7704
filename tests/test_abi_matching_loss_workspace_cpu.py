"""Workspace sizes of the matching loss: each direction asks for what it uses."""
import pytest

from test_abi_network_cpu import L, _loss  # noqa: F401  (L is a fixture)

SIZE = {0: 4, 1: 2, 2: 2}
CASES = [(1, 1, 1, 0), (1, 1000, 24, 0), (16, 44000, 24, 1), (1, 16384, 64, 2), (64, 1 << 20, 24, 1), (64, 1 << 20, 33, 2), (1 << 16, 1 << 24, 24, 1),
         (1, 1 << 24, 128, 0)]


@pytest.mark.parametrize("B,P,d,dtype", CASES)
def test_gradient_holds_rows_and_parts_only(L, B, P, d, dtype):  # noqa: F811
    """Rows as copied, and where they are not written directly (d not a multiple of 4, or up to 16 pieces of few matches) their parts."""
    dp = 32 if d <= 32 else 64 if d <= 64 else 128
    n = L.ddm_matching_loss_backward_workspace_bytes(B, P, d, dtype)
    pieces = 16 if P < 1 << 16 else 0 if d % 4 == 0 else 1
    assert 256 <= n <= 2 * P * dp * SIZE[dtype] + 2 * pieces * P * dp * 4 + 1024
    both = L.ddm_matching_loss_workspace_bytes(B, P, d, dtype)
    assert both == max(n, L.ddm_matching_loss_forward_workspace_bytes(B, P, d, dtype))


def test_each_direction_refuses_less_than_its_own(L):  # noqa: F811
    f = L.ddm_matching_loss_forward_workspace_bytes(2, 50000, 24, 1)
    b = L.ddm_matching_loss_backward_workspace_bytes(2, 50000, 24, 1)
    assert b < f
    assert _loss(L, P=50000, wsb=f - 1) == -3
    assert _loss(L, backward=True, P=50000, wsb=b - 1) == -3


@pytest.mark.parametrize("bad", [(0, 8, 24, 1), (1, -1, 24, 1), (1, (1 << 24) + 1, 24, 1), (1, 8, 0, 1), (1, 8, 129, 1), (1, 8, 24, 3)])
def test_sizes_that_are_refused_have_none(L, bad):  # noqa: F811
    assert L.ddm_matching_loss_forward_workspace_bytes(*bad) == 0 and L.ddm_matching_loss_backward_workspace_bytes(*bad) == 0


def test_forward_sums_stay_small_beside_the_card(L):  # noqa: F811
    """Rows as copied, 640 bytes a match of sums up to 2^18 matches, half a kilobyte beyond, and never more than 1 GiB of them."""
    for P in (4096, 1 << 18, (1 << 18) + 1, 1 << 19, 1 << 20, 1 << 22, (1 << 22) + 1, 1 << 24):
        for B in (1, 64):
            n = L.ddm_matching_loss_forward_workspace_bytes(B, P, 24, 1) - 2 * P * 32 * 2
            other = (2 * 16 * 8 if P < 1 << 16 else 2 * 8) * P + 4 * P + 16 * (P // 128 + B + 2) + 2048
            assert n <= (640 if P <= 1 << 18 else 384) * P + other
            assert n <= (1 << 30) + other
