"""The range of float16 in the gated layer's gradient. The projections' gradients may lie anywhere: they are held in units of the largest.
Projections beyond 65504 are kept as infinite, as is documented, and reach what they are part of and nothing else; bfloat16 does not have
that limit. h, which is formed from 32-bit projections, is right throughout."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("rows", [6, 90])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_projection_beyond_float16(ddm, dtype, rows):
    cols, hidden, row, unit = 24, 20, 4, 7
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    x, w = torch.randn(rows, cols, generator=g, device="cuda"), torch.randn(2 * hidden, cols, generator=g, device="cuda")
    x[:, 0], w[:, 0] = 0, 0
    x[row, 0], w[hidden + unit, 0], w[unit, 0] = 1000, 1000, 0.002       # u = 10^6, g = 2 and a little
    x, w, dh = x.to(dtype), w.to(dtype), (1e-3 * torch.randn(rows, hidden, generator=g, device="cuda")).to(dtype)
    h, kept = ddm.gated_linear_forward(x, w, activation="sigmoid", keep=True)
    dx, dw, db = ddm.gated_linear_backward(dh, x, w, kept, activation="sigmoid")
    p = x.double() @ w.double().T
    want = torch.sigmoid(p[:, :hidden]) * p[:, hidden:]
    there = want.abs() < 65504
    assert not there[row, unit] and there.sum() == rows * hidden - 1
    eps = torch.finfo(dtype).eps
    assert ((h.double() - want).abs() <= eps * want.abs() + 1e-6)[there].all()
    if dtype == torch.bfloat16:
        assert all(torch.isfinite(t).all() for t in (h, kept, dx, dw, db))
        return
    assert kept[row, hidden + unit] == float("inf")
    # dx of its row, the gate's weight and bias of its unit; u itself is no part of its own gradient
    lost = torch.zeros(rows, dtype=torch.bool, device="cuda"), torch.zeros(2 * hidden, dtype=torch.bool, device="cuda")
    lost[0][row], lost[1][unit] = True, True
    assert not torch.isfinite(dx[row]).any() and not torch.isfinite(dw[unit, x[row] != 0]).any() and not torch.isfinite(db[unit])
    assert torch.isfinite(dx[~lost[0]]).all() and torch.isfinite(dw[~lost[1]]).all() and torch.isfinite(db[~lost[1]]).all()
    # those others are what they are without that unit's projection beyond range
    x2 = x.clone()
    x2[row, 0] = 0
    h2, kept2 = ddm.gated_linear_forward(x2, w, activation="sigmoid", keep=True)
    dx2 = ddm.gated_linear_backward(dh, x2, w, kept2, activation="sigmoid")[0]
    assert torch.equal(dx[~lost[0]], dx2[~lost[0]])


@pytest.mark.parametrize("rows,value,size,dh", [
    (1000, 4.0, 0.25, 2.0 ** -22),          # gradients of projections among float16's smallest numbers
    (70000, 2.0 ** -7, 2.0 ** -12, 2.0 ** -20),   # below them, many of which are something
    (40, 1024.0, 2.0 ** -10, 1000.0),       # beyond its largest, in sums that are not
    (3, 1024.0, 2.0 ** -10, 1000.0)])
def test_gradients_of_projections_anywhere(ddm, rows, value, size, dh):
    """All terms are positive and g = u = value exactly, so an error is that of the roundings alone, relative to the result: those of dg
    and du to the type (u = 2^-11), of the result (u, half of the smallest step at least), sums of K terms in 32 bits (K + 64) E."""
    E, u, cols, hidden = 2.0 ** -24, 2.0 ** -11, 32, 24
    x = torch.full((rows, cols), value / size / cols, device="cuda").half()
    w = torch.full((2 * hidden, cols), size, device="cuda").half()
    d = torch.full((rows, hidden), dh, device="cuda").half()
    h, kept = ddm.gated_linear_forward(x, w, keep=True)
    assert (kept == value).all() and (d == dh).all()
    dx, dw, db = ddm.gated_linear_backward(d, x, w, kept)
    t = torch.sigmoid(torch.tensor(value, dtype=torch.float64)).item()
    dg, du = dh * value * t * (1 + value * (1 - t)), dh * value * t
    assert min(dg, du) < 2.0 ** -17 or max(dg, du) > 65504
    for got, want, terms in ((dx, hidden * size * (dg + du), 2 * hidden), (dw[:hidden], rows * dg * x[0, 0].item(), rows),
                             (dw[hidden:], rows * du * x[0, 0].item(), rows), (db[:hidden], rows * dg, rows), (db[hidden:], rows * du, rows)):
        if want > 65504:
            assert (got == float("inf")).all()
        else:
            assert ((got.double() - want).abs() <= (2.1 * u + (terms + 64) * E) * want + 2.0 ** -25).all(), (got.flatten()[0].item(), want)


def test_units_follow_the_data(ddm):
    """Gradients of one captured step, replayed with outputs' gradients of any size, are those of size one times that power of two."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, d = r(130, 40).half(), (r(2 * 24, 40) / 6).half(), r(130, 24).half()
    d[d.abs() < 2.0 ** -4] = 0                                   # all of d / 2^10 is a normal number
    dh = d.clone()
    _, kept = ddm.gated_linear_forward(x, w, keep=True)
    ddm.gated_linear_backward(dh, x, w, kept)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ddm.gated_linear_backward(dh, x, w, kept)
    want = [t.float() for t in ddm.gated_linear_backward(d, x, w, kept)]
    for power in (0, -10, 4, -6, 8, 0, -9):
        dh.copy_(d.float() * 2.0 ** power)
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            b = b * 2.0 ** power
            # both are rounded once (2 * 2^-11, half a smallest step at least); where no unit was needed, projections' gradients were
            # off by up to 2^-25 each, in sums of at most 130 of them times inputs below 4
            there = b.abs() < 60000
            slack = 2.0 ** -24 + 2.0 ** -25 * max(2.0 ** power, 1) * 130 * 4 + 2.0 ** -10 * b.abs()
            assert ((a.float() - b).abs() <= slack)[there].all(), power
