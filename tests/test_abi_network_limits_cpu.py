"""The last accepted and the first refused value of each limit on sizes. Workspace sizes answer for the accepted ones, so nothing is
launched; fake pointers are never touched."""
import pytest

from test_abi_network_cpu import L, _attn, _loss, _norm, _norm_back  # noqa: F401  (L is a fixture)

ROWS = (1 << 31) - 4097                                  # rows (tokens times a group's heads)
KEYS = (1 << 31) - 1 - (1 << 22) - 1
HALF = ((1 << 23) - 4) * 128 + 127                       # rows or keys of each of two key heads, one sequence
ATTENTION = [(dict(B=1 << 20, Tq=8, Tk=8, Hq=1, Hkv=1), dict(B=(1 << 20) + 1, Tq=8, Tk=8, Hq=1, Hkv=1)),
             (dict(B=1, Tq=ROWS, Tk=8, Hq=1, Hkv=1), dict(B=1, Tq=ROWS + 1, Tk=8, Hq=1, Hkv=1)),
             (dict(B=1, Tq=ROWS // 71, Tk=8, Hq=71, Hkv=1), dict(B=1, Tq=ROWS // 71 + 1, Tk=8, Hq=71, Hkv=1)),
             (dict(B=1, Tq=131072, Tk=131072, Hq=128, Hkv=1), None),
             (dict(B=1, Tq=ROWS // 128, Tk=8, Hq=128, Hkv=1), dict(B=1, Tq=ROWS // 128 + 1, Tk=8, Hq=128, Hkv=1)),
             (dict(B=1, Tq=8, Tk=KEYS, Hq=1, Hkv=1), dict(B=1, Tq=8, Tk=KEYS + 1, Hq=1, Hkv=1)),
             (dict(B=1, Tq=HALF, Tk=8, Hq=2, Hkv=2), dict(B=1, Tq=HALF + 1, Tk=8, Hq=2, Hkv=2)),
             (dict(B=1, Tq=8, Tk=HALF, Hq=2, Hkv=2), dict(B=1, Tq=8, Tk=HALF + 1, Hq=2, Hkv=2)),
             (dict(B=16, Tq=8, Tk=8, Hq=932067, Hkv=932067), dict(B=16, Tq=8, Tk=8, Hq=932068, Hkv=932068))]


@pytest.mark.parametrize("last,refused", ATTENTION)
def test_attention(L, last, refused):  # noqa: F811
    f, b = L.ddm_attention_forward_workspace_bytes, L.ddm_attention_backward_workspace_bytes
    sizes = lambda a: (a["B"], a["Tq"], a["Tk"], a["Hq"], a["Hkv"], 64, 1)  # noqa: E731
    assert f(*sizes(last)) > 0 and b(*sizes(last)) > 0
    if refused:
        assert f(*sizes(refused)) == 0 and b(*sizes(refused)) == 0
        assert _attn(L, **refused) == -1 and _attn(L, backward=True, **refused) == -1


def test_attention_strides(L):  # noqa: F811
    """A token stride of 16 MB, and a group's heads over 512 MB, are the first refused ones; the ones below fail only for the
    workspace, which is looked at last."""
    e = 2
    for s, status in (((1 << 24) // e - 8, -3), ((1 << 24) // e, -1)):
        assert _attn(L, Tq=1, Tk=5000, Hq=2, kt=s, ws=None) == status
        assert _attn(L, backward=True, kt=s, ws=None) == status
    for s, status in (((1 << 29) // 2 // e - 8, -3), ((1 << 29) // 2 // e, -1)):
        assert _attn(L, backward=True, qh=s, ws=None) == status
        assert _attn(L, backward=True, gh=s, ws=None) == status


def test_layer_norm(L):  # noqa: F811
    w = L.ddm_layer_norm_backward_workspace_bytes
    assert w((1 << 31) - 1, 8192, 2) > 0 and w(1 << 31, 8192, 2) == 0 and w(10, 8193, 2) == 0
    assert _norm(L, N=1 << 31) == -1 and _norm_back(L, N=1 << 31) == -1


@pytest.mark.parametrize("last,refused", [((1, 1 << 24, 128, 0), (1, (1 << 24) + 1, 128, 0)), ((1 << 20, 8, 8, 1), ((1 << 20) + 1, 8, 8, 1))])
def test_matching_loss(L, last, refused):  # noqa: F811
    assert L.ddm_matching_loss_workspace_bytes(*last) > 0 and L.ddm_matching_loss_workspace_bytes(*refused) == 0
    change = dict(zip(("B", "P", "d", "dtype"), refused))
    assert _loss(L, **change) == -1 and _loss(L, backward=True, **change) == -1
