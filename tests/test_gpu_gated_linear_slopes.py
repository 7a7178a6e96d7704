"""The gated layer's activations and their slopes over a range of the gate's projection, each against 64 bits and relative to its own
size, so that tails keep their digits. One input of one makes the weight the projections: h = act(g) u, and with u = dh = 1 the
weight's gradient is act'(g) for the gate's rows and act(g) for the others.

Tolerances with E = 2^-24. Sigmoid: exp(-g) is off by (|g| + 2) 2 E (argument and exponential), 1 / (1 + exp) by as much at most and 3 E,
and the derivative, sigmoid(g) sigmoid(-g), has two of those: (|g| + 2) 4 E + 10 E, for the value half of it.

GELU: Phi(-|g|) is a product of an exponential whose argument is carried in twice 32 bits (4 E), a reciprocal (3 E) and a polynomial of it
(1.6 E off by itself; its nine steps, whose terms come to at most 2.2 of its value, 12 E, the reciprocal's error 6 E): with the products 32 E.
The slope is its sum with g times the density, each off by that of its own size. Below 2^-126 results may be zero."""
import math
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


def measured(ddm, g, kind, rows):
    """act and act' at g: from h and, with one row, the weight's gradient; from more rows also the path for many rows."""
    one = torch.ones_like(g)
    x, w = torch.ones(rows, 1, device="cuda"), torch.cat((g, one))[:, None].contiguous()
    h, kept = ddm.gated_linear_forward(x, w, activation=kind, keep=True)
    assert (kept[:, :len(g)] == g).all() and (h == h[0]).all()
    dw = ddm.gated_linear_backward(torch.ones(1, len(g), device="cuda"), x[:1], w, kept[:1].contiguous(), activation=kind)[1][:, 0]
    assert torch.equal(dw[len(g):], h[0])
    return h[0].double(), dw[:len(g)].double()


@pytest.mark.parametrize("rows", [1, 100])
def test_sigmoid(ddm, rows):
    g = torch.cat((torch.linspace(-80, 80, 4001), torch.tensor([5.0, 8.0, 10.0, 12.0, 16.0, 17.0, 20.0, -17.0, 0.0, -0.0]))).cuda()
    act, slope = measured(ddm, g, "sigmoid", rows)
    G = g.double()
    t = torch.sigmoid(G)
    assert ((act - t).abs() <= ((G.abs() + 2) * 2 * E + 5 * E) * t).all()
    want = t * torch.sigmoid(-G)
    assert ((slope - want).abs() <= ((G.abs() + 2) * 4 * E + 10 * E) * want).all()


@pytest.mark.parametrize("rows", [1, 100])
def test_gelu(ddm, rows):
    g = torch.cat((torch.linspace(-13, 13, 26001), torch.tensor([-20.0, -1e4, -1e30, 1e4, 0.0, -0.0]))).cuda()
    act, slope = measured(ddm, g, "gelu", rows)
    G = g.double()
    phi = 0.5 * torch.special.erfc(-G / math.sqrt(2))
    density = torch.exp(-G * G / 2) / math.sqrt(2 * math.pi)
    tiny = 13 * 2.0 ** -126
    assert ((act - G * phi).abs() <= 32 * E * (G * phi).abs() + tiny).all()
    assert ((slope - (phi + G * density)).abs() <= 32 * E * (phi + (G * density).abs()) + tiny).all()
