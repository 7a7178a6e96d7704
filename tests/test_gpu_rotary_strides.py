"""Strides of a rotary call: an only token's or head's says nothing and may be any number, as torch leaves it after slicing."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("far", [0, 3, 1 << 41, (1 << 62) - 1])
def test_only_tokens_and_heads(ddm, far, interleaved):
    f = ddm.rotary_frequencies(8, device="cuda")
    x = torch.randn(12, 3, 16, device="cuda").bfloat16()
    pos = torch.arange(12, dtype=torch.int32, device="cuda")
    how = dict(interleaved=interleaved)
    want, _ = ddm.rotary_forward(x, None, pos, f, **how)
    # one token of three heads, twelve tokens of one head, one of one; as queries, as keys and as outputs
    for shape, strides, at, p, w in (((1, 3, 16), (far, 16, 1), x[5], pos[5:6], want[5:6]),
                                     ((12, 1, 16), (48, far, 1), x[:, 1], pos, want[:, 1:2]),
                                     ((1, 1, 16), (far, far, 1), x[7, 2], pos[7:8], want[7:8, 2:3])):
        view = at.as_strided(shape, strides)
        a, b = ddm.rotary_forward(view, view, p, f, **how)
        assert torch.equal(a, w) and torch.equal(b, w)
        room = torch.zeros_like(x)
        out = room.as_strided(shape, strides)
        a, _ = ddm.rotary_forward(w, None, p, f, out=(out, None), **how)
        assert torch.equal(a, ddm.rotary_forward(w, None, p, f, **how)[0])
