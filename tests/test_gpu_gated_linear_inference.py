"""Inference through the differentiable gated layer is the plain call: no projections are kept, and memory shows it."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


def peak(call):
    """Bytes that the call asked for at most. (What it is given also depends on the blocks that are free.)"""
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["requested_bytes.all.current"]
    torch.cuda.reset_peak_memory_stats()
    out = call()
    torch.cuda.synchronize()
    return torch.cuda.memory_stats()["requested_bytes.all.peak"] - before, out


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("rows", [1, 600])
def test_no_more_memory_than_the_plain_call(ddm, mode, rows):
    x = torch.randn(rows, 512, device="cuda").bfloat16()
    w = torch.nn.Parameter((torch.randn(2 * 1040, 512, device="cuda") / 22).bfloat16())
    b = torch.nn.Parameter(torch.randn(2 * 1040, device="cuda").bfloat16())
    with mode():
        plain, want = peak(lambda: ddm.gated_linear_forward(x, w, b)[0])
        got, h = peak(lambda: ddm.gated_linear(x, w, b))
    assert torch.equal(h, want) and not h.requires_grad
    assert got == plain
    kept, h = peak(lambda: ddm.gated_linear(x, w, b))
    assert torch.equal(h, want) and h.requires_grad and kept == plain + rows * 2 * 1040 * 2
    h.float().sum().backward()
    assert w.grad.shape == w.shape and b.grad.shape == b.shape


@pytest.mark.parametrize("rows", [20, 600])
def test_no_room_for_a_copy_that_is_not_made(ddm, rows):
    """x on whole 16-byte pieces takes no workspace for its copy; off them it does, and gives the same."""
    cols, hidden = 512, 40
    odd = torch.randn(rows * cols + 1, device="cuda").half()[1:].view(rows, cols)
    x, w = odd.clone(), (torch.randn(2 * hidden, cols, device="cuda") / 22).half()
    dh = torch.randn(rows, hidden, device="cuda").half()
    whole, (h, kept) = peak(lambda: ddm.gated_linear_forward(x, w, keep=True))
    copied, (g, _) = peak(lambda: ddm.gated_linear_forward(odd, w, keep=True))
    assert torch.equal(h, g) and copied >= whole + rows * cols * 2 - 16 and whole < copied
    whole, got = peak(lambda: ddm.gated_linear_backward(dh, x, w, kept))
    copied, want = peak(lambda: ddm.gated_linear_backward(dh, odd, w, kept))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and copied >= whole + rows * cols * 2
