"""The gated layer's workspace for an x whose rows are whole 16-byte pieces, and for others. Host checks alone: addresses are made up, and
every call is refused for its workspace."""
import os

import pytest

FAKE = 1 << 40


@pytest.fixture(scope="module")
def L():
    import dense_descriptor_matching_amd as ddm
    if not os.path.exists(ddm.LIB_PATH):
        pytest.fail("libddm.so not built: run __graft_entry__.build()")
    return ddm.lib()


def calls(L, x, ldx, N, C, F, dtype, nbytes):
    return (L.ddm_gated_linear_forward(x, ldx, FAKE, None, N, C, F, dtype, 0, FAKE, None, FAKE, nbytes[0], None),
            L.ddm_gated_linear_backward(FAKE, x, ldx, FAKE, FAKE, N, C, F, dtype, 0, FAKE, FAKE, FAKE, FAKE, nbytes[1], None))


@pytest.mark.parametrize("dtype,e", [(0, 4), (1, 2), (2, 2)])
@pytest.mark.parametrize("N,C,F", [(1, 64, 48), (20, 1024, 100), (3000, 512, 1000), (24576, 1024, 2736)])
def test_a_copy_of_x_only_where_it_is_made(L, N, C, F, dtype, e):
    full = [f(N, C, F, dtype) for f in (L.ddm_gated_linear_forward_workspace_bytes, L.ddm_gated_linear_backward_workspace_bytes)]
    copy = L.ddm_gated_linear_repack_bytes(N, C, dtype)
    assert N * C * e <= copy < N * C * e + 256
    for x, ldx in ((FAKE + e, C), (FAKE + 8, C)) + (((FAKE, C + 1),) if N > 1 else ()):
        assert calls(L, x, ldx, N, C, F, dtype, [n - 1 for n in full]) == (-3, -3)
    less = [max(n - copy, 16) - 1 for n in full]
    assert calls(L, FAKE, C, N, C, F, dtype, less) == (-3, -3)
    assert calls(L, FAKE, C + 64, N, C, F, dtype, less) == (-3, -3)
    assert [n - copy for n in full][1] >= 2 * N * F * e          # the projections' gradients


def test_sizes_outside_the_limits(L):
    f = L.ddm_gated_linear_repack_bytes
    assert f(-1, 64, 1) == 0 and f(10, 0, 1) == 0 and f(10, 64, 5) == 0 and f((1 << 24) + 1, 64, 1) == 0 and f(0, 64, 1) == 0
