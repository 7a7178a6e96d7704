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
