"""Rotary positions written over tensors that autograd follows: refused where a gradient would be lost, and seen by the
backward passes that were to read what was written over."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


@pytest.fixture
def places(ddm):
    return torch.arange(6, dtype=torch.int32, device="cuda"), ddm.rotary_frequencies(8, device="cuda")


def heads(n=2, **kw):
    return torch.randn(6, n, 16, device="cuda", **kw)


def test_out_with_a_gradient_is_refused(ddm, places):
    q, k, plain = heads(requires_grad=True), heads(1), heads()
    for turn in (ddm.rotary_forward, ddm.rotary_backward):
        for given, key, out in ((q * 1, None, None), (plain, None, (q * 1, None)), (q * 1, k, (plain, k)), (q, None, (plain, None)),
                                (plain, k, (plain, heads(1, requires_grad=True) * 1))):
            with pytest.raises(RuntimeError, match="gradient"):
                turn(given, key, *places, out=(given, key) if out is None else out)
    # without a gradient, or with gradients off, it is what it is without out=
    want, _ = ddm.rotary_forward(plain, None, *places)
    with torch.no_grad():
        v = q * 1
        v.copy_(plain)
        assert torch.equal(ddm.rotary_forward(v, None, *places, out=(v, None))[0], want)
        leaf = plain.clone().requires_grad_()
        assert torch.equal(ddm.rotary_forward(leaf, None, *places, out=(leaf, None))[0], want)
    with torch.inference_mode():
        v = plain.clone()
        assert torch.equal(ddm.rotary_forward(v, None, *places, out=(v, None))[0], want)
    assert torch.equal(ddm.rotary_forward(plain, None, *places, out=(plain, None))[0], want)


def test_what_was_saved_for_a_gradient_is_guarded(ddm, places):
    for which in (0, 1):
        a, v = heads(requires_grad=True), heads()
        y = (a * v).sum()                   # keeps v
        q, k = (v, heads(1)) if which == 0 else (heads(1), v)
        ddm.rotary_forward(q, k, *places, out=iter((q, k)))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    a, v = heads(requires_grad=True), heads()
    y = (a * v).sum()
    ddm.rotary_forward(v, None, *places)    # to tensors of its own: nothing changed
    y.backward()
    assert torch.equal(a.grad, v)
