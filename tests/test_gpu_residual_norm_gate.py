"""The gate's gradient keeps its digits however far the gate is open or shut. Without dy, dx is ds, and dgate = ds scale t o', o' the
derivative of sigmoid, in 64 bits sigmoid(g) sigmoid(-g).

Tolerance, relative, with E = 2^-24 and u the type's unit roundoff: o' = e / (1 + e)^2 with e = exp(-|g|). The argument times log2(e) and
the exponential leave e off by (|g| + 2) 2 E; the two reciprocals of 1 + e add as much again at most and 3 E each, the products
with ds, scale and t E each: (|g| + 2) 4 E + 10 E; then one rounding to the type, half of float16's smallest step at least."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("cols", [321, 1600, 5000])
def test_far_open_and_shut(dtype, cols):
    import dense_descriptor_matching_amd as ddm
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    far = 80.0 if dtype != torch.float16 else 12.0          # of float16's steps some are left
    gate = torch.linspace(-far, far, 4 * cols, device="cuda").view(cols, 4).t().contiguous().to(dtype)
    x, t, ds = (torch.randn(4, cols, generator=g, device="cuda").to(dtype) for _ in range(3))
    scale = 0.5 + torch.rand(cols, generator=g, device="cuda")
    s, _, stats = ddm.residual_norm_forward(x, t, scale=scale, gate=gate)
    dx, _, _, _, _, dgate = ddm.residual_norm_backward(None, ds, x, t, stats, scale=scale, gate=gate)[:6]
    assert torch.equal(dx, ds)
    G = gate.double()
    want = ds.double() * scale.double() * t.double() * torch.sigmoid(G) * torch.sigmoid(-G)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    off = (dgate.double() - want).abs() - tiny - ((G.abs() + 2) * 4 * E + 10 * E + U[dtype]) * want.abs()
    assert off.max().item() <= 0, off.max().item()
