"""The gated linear layer against its definition in 64 bits.

With u the unit roundoff of the type (2^-8 bfloat16, 2^-11 float16, 2^-24 float32) and E = 2^-24. Bounds per element: a product of K
terms accumulated in 32 bits is off by at most (K + 8) E of its absolute terms (16-bit products are exact). The activations' slopes are
below 1.13 and their second derivatives below 0.8; their own evaluation is off by (|g| + 8) 4 E of what it comes to, and of the slope
by (|g| + 8) 4 E. g and u are rounded to the type before the gradient takes them and dg and du before the products: each adds u of its
value.

Such bounds add every rounding with its worst sign, so the error's norm is held too: independent roundings of relative size up to u are
u / sqrt(3) in the mean square at most (a rounding is off by u only at the bottom of a binade). Behind dx and dweight lie those of g, of u,
of dg or du and the output's own; those of g enter through act' and act'', at most |g| 0.8 + 1.13 < 3 times for the |g| < 3 that matter, but on
half of the terms: sqrt(3 + 3) u / sqrt(3) < 1.5 u; the tests ask for 1.5 u, or in 32 bits, where sums dominate, for 64 E.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
E = 2.0 ** -24


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


def make(rows, cols, hidden, dtype, bias=True, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, dh = r(rows, cols), r(2 * hidden, cols) / math.sqrt(cols), r(rows, hidden)
    b = 0.3 * r(2 * hidden) if bias else None
    return tuple(None if t is None else t.to(DT[dtype]) for t in (x, w, b, dh))


def activation(g, kind):
    if kind == "gelu":
        phi = torch.special.ndtr(g)
        return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    t = torch.sigmoid(g)
    return (t, t * (1 - t)) if kind == "sigmoid" else (g * t, t * (1 + g * (1 - t)))


def expected(x, w, b, dh, kind, dtype):
    x, w, dh = x.double(), w.double(), dh.double()
    n, c = x.shape
    f = len(w) // 2
    u, tiny = U[dtype], TINY[dtype]
    p, size = x @ w.T, (c + 8) * E * (x.abs() @ w.abs().T)
    if b is not None:
        p = p + b.double()
        size = size + E * p.abs()
    g, v, g_err, v_err = p[:, :f], p[:, f:], size[:, :f], size[:, f:]
    a, slope = activation(g, kind)
    a_err = 1.13 * g_err + (g.abs() + 8) * 4 * E * a.abs()
    want = dict(h=a * v)
    tol = dict(h=u * (a * v).abs() + tiny + a_err * v.abs() + a.abs() * v_err + a_err * v_err + E * (a * v).abs())
    # g and v as they are kept
    g_err, v_err = g_err + u * g.abs() + tiny, v_err + u * v.abs() + tiny
    a_err = 1.13 * g_err + (g.abs() + 8) * 4 * E * a.abs()
    s_err = 0.8 * g_err + (g.abs() + 8) * 4 * E
    dg, dv = dh * v * slope, dh * a
    dg_err = dh.abs() * (v.abs() * s_err + slope.abs() * v_err + s_err * v_err) + 2 * E * dg.abs()
    dv_err = dh.abs() * a_err + E * dv.abs()
    want["dbias"] = torch.cat((dg.sum(0), dv.sum(0)))
    tol["dbias"] = u * want["dbias"].abs() + tiny + torch.cat((dg_err.sum(0), dv_err.sum(0))) + (n + 40) * E * torch.cat(
        (dg.abs().sum(0), dv.abs().sum(0)))
    d, d_err = torch.cat((dg, dv), 1), torch.cat((dg_err, dv_err), 1)
    d_err = d_err + u * d.abs() + tiny
    want["dx"], want["dweight"] = d @ w, d.T @ x
    tol["dx"] = u * want["dx"].abs() + tiny + d_err @ w.abs() + (2 * f + 8) * E * (d.abs() @ w.abs())
    tol["dweight"] = u * want["dweight"].abs() + tiny + d_err.T @ x.abs() + (n + 8) * E * (d.abs().T @ x.abs())
    return want, tol


def run(ddm, x, w, b, dh, kind):
    h, kept = ddm.gated_linear_forward(x, w, b, activation=kind, keep=True)
    dx, dw, db = ddm.gated_linear_backward(dh, x, w, kept, activation=kind)
    return dict(h=h, dx=dx, dweight=dw, dbias=db)


def check(ddm, args, kind, dtype):
    got = run(ddm, *args, kind)
    want, tol = expected(*args, kind, dtype)
    for name in want:
        off = (got[name].double() - want[name]).abs() - 1.25 * tol[name]
        assert not torch.isnan(off).any(), name
        assert off.max().item() <= 0, (name, off.max().item())
        # a norm is one where there are elements enough
        if want[name].numel() >= 4096:
            norm = ((got[name].double() - want[name]).norm() / want[name].norm()).item()
            assert norm <= (64 * E if dtype == "f32" else 1.5 * U[dtype]), (name, norm)
    h, none = ddm.gated_linear_forward(args[0], args[1], args[2], activation=kind)
    assert none is None and torch.equal(h, got["h"])


SIZES = [(1, 1, 1), (1, 64, 16), (2, 1024, 272), (3, 7, 5), (5, 130, 33), (31, 64, 100), (32, 96, 64), (33, 200, 65), (64, 513, 47),
         (65, 64, 64), (100, 1000, 24), (127, 40, 129), (128, 128, 128), (129, 264, 136), (300, 771, 130), (513, 64, 257), (1000, 8, 8),
         (70, 4104, 40), (2049, 72, 520), (9000, 64, 24)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,hidden", SIZES)
def test_values_and_gradients(ddm, dtype, rows, cols, hidden):
    kind = ("silu", "gelu", "sigmoid")[(rows + cols) % 3]
    check(ddm, make(rows, cols, hidden, dtype, bias=hidden % 2 == 0, seed=rows), kind, dtype)


@pytest.mark.parametrize("kind", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_activations(ddm, dtype, kind):
    check(ddm, make(200, 128, 96, dtype, seed=5), kind, dtype)
    check(ddm, make(20, 128, 96, dtype, seed=6), kind, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols,hidden", [(4096, 512, 2100), (2100, 1032, 4096)])
def test_large_tiles(ddm, dtype, rows, cols, hidden):
    """Products of many tiles; whole and part tiles on every side."""
    check(ddm, make(rows, cols, hidden, dtype, seed=7), "silu", dtype)


def test_projections_far_from_zero(ddm):
    """Activations of projections where exponentials over- and underflow."""
    x = torch.ones(8, 8, device="cuda")
    w = torch.zeros(2 * 8, 8, device="cuda")
    w[:8, 0] = torch.tensor([-3e4, -200.0, -100.0, -30.0, 30.0, 100.0, 200.0, 3e4])
    w[8:, 0] = 2.0
    for kind, want in (("silu", [0, 0, 0, None, 60, 200, 400, 6e4]), ("gelu", [0, 0, 0, 0, 60, 200, 400, 6e4]),
                       ("sigmoid", [0, 0, 0, None, 2, 2, 2, 2])):
        for dtype in ("f32", "bf16"):
            got = run(ddm, x.to(DT[dtype]), w.to(DT[dtype]), None, x.to(DT[dtype]), kind)
            assert all(torch.isfinite(t).all() for t in got.values())
            for i, v in enumerate(want):
                if v is not None:
                    assert abs(got["h"][0, i].item() - v) <= abs(v) * 2 * U[dtype] + 1e-35, (kind, i)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [20, 200])
def test_row_strides_and_odd_addresses(ddm, dtype, rows):
    """Views give what their copies give, with rows on 16-byte boundaries and off them; beside them stands NaN."""
    for cols, ld, first in ((64, 96, 0), (64, 96, 3), (64, 99, 0), (61, 64, 0), (61, 77, 1)):
        x, w, b, dh = make(rows, cols, 40, dtype, seed=8)
        want = run(ddm, x, w, b, dh, "silu")
        wide = torch.full((rows * ld + 8,), float("nan"), device="cuda", dtype=DT[dtype])[first:first + rows * ld].view(rows, ld)
        view = wide[:, :cols].copy_(x)
        odd_b = torch.empty(81, device="cuda", dtype=DT[dtype])[1:].copy_(b)
        odd_dh = torch.empty(rows * 40 + 1, device="cuda", dtype=DT[dtype])[1:].view(rows, 40).copy_(dh)
        got = run(ddm, view, w, odd_b, odd_dh, "silu")
        for n in want:
            assert torch.equal(got[n], want[n]), (n, cols, ld, first)


def test_nan_stays_in_its_row(ddm):
    for rows in (30, 150):
        x, w, b, dh = make(rows, 72, 50, "bf16", seed=9)
        clean = run(ddm, x, w, b, dh, "silu")
        x = x.clone()
        x[11, 3] = float("nan")
        got = run(ddm, x, w, b, dh, "silu")
        keep = [i for i in range(rows) if i != 11]
        for n in ("h", "dx"):
            assert torch.equal(got[n][keep], clean[n][keep]) and torch.isnan(got[n][11]).all()


def test_no_rows_and_leading_dimensions(ddm):
    x, w, b, dh = make(6, 32, 24, "f16", seed=10)
    h, kept = ddm.gated_linear_forward(x[:0], w, b, keep=True)
    assert h.shape == (0, 24) and kept.shape == (0, 48)
    dx, dw, db = ddm.gated_linear_backward(h, x[:0], w, kept)
    assert dx.shape == (0, 32) and (dw == 0).all() and (db == 0).all() and dw.shape == w.shape
    h3, _ = ddm.gated_linear_forward(x.view(2, 3, 32), w, b)
    assert h3.shape == (2, 3, 24) and torch.equal(h3.view(6, 24), ddm.gated_linear_forward(x, w, b)[0])


@pytest.mark.parametrize("rows", [40, 700])
def test_parts_repeats_streams(ddm, rows):
    x, w, b, dh = make(rows, 520, 264, "bf16", seed=11)
    _, kept = ddm.gated_linear_forward(x, w, b, keep=True)
    full = ddm.gated_linear_backward(dh, x, w, kept)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = ddm.gated_linear_backward(dh, x, w, kept)
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(full, again))
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        got = ddm.gated_linear_backward(dh, x, w, kept, need_dx=need[0], need_dweight=need[1], need_dbias=need[2])
        for g, t, n in zip(got, full, need):
            assert torch.equal(g, t) if n else g is None


@pytest.mark.parametrize("rows", [3, 500])
def test_graph_replays(ddm, rows):
    args = make(rows, 333, 130, "bf16", seed=12)
    want = run(ddm, *args, "gelu")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ddm, *args, "gelu")
    for _ in range(3):
        for t in got.values():
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("kind", ["silu", "gelu", "sigmoid"])
def test_autograd_and_differences(ddm, kind):
    """Differences in 64 bits of the definition agree with autograd's float32 gradient to its rounding."""
    x, w, b, dh = make(9, 20, 14, "f32", seed=13)
    t = [v.clone().requires_grad_() for v in (x, w, b)]
    (ddm.gated_linear(*t, activation=kind) * dh).sum().backward()

    def f(x, w, b):
        g, v = (x @ w.T + b).chunk(2, dim=1)
        return (activation(g, kind)[0] * v * dh.double()).sum()

    base = [v.double() for v in (x, w, b)]
    for i in range(3):
        d = torch.randn_like(base[i])
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + 1e-4 * d, base[i] - 1e-4 * d
        diff = (f(*up) - f(*down)) / 2e-4
        assert abs(diff - (t[i].grad.double() * d).sum()) <= 1e-4 * (1 + t[i].grad.double().norm() * d.norm()), i
    with torch.no_grad():
        assert torch.equal(ddm.gated_linear(*t, activation=kind), ddm.gated_linear_forward(x, w, b, activation=kind)[0])
    z = x.clone().requires_grad_()
    ddm.gated_linear(z, w, activation=kind).sum().backward()
    assert z.grad.shape == x.shape


def test_refusals(ddm):
    x, w, b, dh = make(6, 32, 24, "f16")
    f = ddm.gated_linear_forward
    for bad in ((x.cpu(), w), (x.double(), w.double()), (x, w.float()), (x, w, b.float())):
        with pytest.raises((TypeError, ValueError)):
            f(*bad)
    for bad in ((x, w[:47]), (x, w[:, :31].contiguous()), (x, w[0]), (x, w.t()), (x, w, b[:47]), (x.t(), w[:, :6].contiguous())):
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(ValueError):
        f(x, w, activation="relu")
    with pytest.raises(ddm.DDMError) as e:               # a weight off a 16-byte boundary
        f(x, torch.empty(48 * 32 + 1, device="cuda", dtype=torch.float16)[1:].view(48, 32))
    assert e.value.status == -1
    h, kept = f(x, w, b, keep=True)
    g = ddm.gated_linear_backward
    for bad in ((dh[:5], x, w, kept), (dh.t(), x, w, kept), (dh, x, w, kept[:, :47])):
        with pytest.raises(ValueError):
            g(*bad)
    for bad in ((dh.float(), x, w, kept), (dh, x, w, kept.float()), (dh, x, w, None)):
        with pytest.raises(TypeError):
            g(*bad)
