"""Rotary outputs that lie over one another are refused; layouts in which they do not are taken, whatever the order of their axes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


def test_one_buffer_for_both_is_refused(ddm):
    f, pos = ddm.rotary_frequencies(8, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda")
    q, k = torch.randn(5, 2, 16, device="cuda"), torch.randn(5, 2, 16, device="cuda")
    room = torch.zeros_like(q)
    flat = torch.zeros(264, device="cuda")
    for out in ((room, room), (k, q), (k, room), (room, q), (flat.as_strided((5, 2, 16), (16, 16, 1)), room),
                (flat.as_strided((5, 2, 16), (24, 12, 1)), room), (flat.as_strided((5, 2, 16), (40, 88, 1)), room)):
        with pytest.raises(ddm.DDMError) as e:
            ddm.rotary_forward(q, k, pos, f, out=out)
        assert e.value.status == -1
    assert (room == 0).all() and (flat == 0).all()


def test_layouts_that_do_not_overlap(ddm):
    f, pos = ddm.rotary_frequencies(8, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda")
    q, k = torch.randn(5, 3, 16, device="cuda"), torch.randn(5, 2, 16, device="cuda")
    want = ddm.rotary_forward(q, k, pos, f)
    # one after another in a row, heads first, with gaps, tokens of a head between those of another
    packed = torch.empty(5, 5, 16, device="cuda")
    for out in ((packed[:, :3], packed[:, 3:]), (packed[:, 2:], packed[:, :2]),
                (torch.empty(3, 5, 16, device="cuda").transpose(0, 1), torch.empty(2, 5, 16, device="cuda").transpose(0, 1)),
                (torch.empty(5, 3, 4, 16, device="cuda")[:, :, 1], torch.empty(5, 2, 4, 16, device="cuda")[:, :, 3]),
                (torch.empty(400, device="cuda").as_strided((5, 3, 16), (32, 80, 1)), torch.empty(400, device="cuda").as_strided(
                    (5, 2, 16), (32, 48, 1)))):
        got = ddm.rotary_forward(q, k, pos, f, out=out)
        assert all(a.data_ptr() == o.data_ptr() and torch.equal(a, w) for a, o, w in zip(got, out, want))
