"""Layer norm against its definition in 64 bits.

Tolerances per element: with u the unit roundoff of an output's type (2^-8 bfloat16, 2^-11 float16, 2^-24 float32) an output
is rounded once, u |value|; the 32-bit sums behind it have relative error (log2 C + 8) 2^-24 of their absolute terms (they
are summed in trees), which reaches xh through the mean by rstd (|x| + mean |x|), and sums over N rows add up to N + 40 roundings.
"""
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


def make(rows, cols, dtype, wtype, seed=0, offset=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return ((r(rows, cols) * r(cols).mul(0.5).exp() + offset * r(cols)).to(DT[dtype]), (1 + 0.2 * r(cols)).to(DT[wtype]),
            (0.2 * r(cols)).to(DT[wtype]), r(rows, cols).to(DT[dtype]))


def check(ddm, x, w, b, dy, dtype, wtype, eps=1e-6):
    y, mean, rstd = ddm.layer_norm_forward(x, w, b, eps=eps)
    dx, dw, db = ddm.layer_norm_backward(dy, x, w, mean, rstd, wtype=DT[wtype])
    X, G = x.double(), dy.double()
    n, c = X.shape
    W = torch.ones(c, dtype=torch.float64, device="cuda") if w is None else w.double()
    Bv = torch.zeros(c, dtype=torch.float64, device="cuda") if b is None else b.double()
    mu = X.mean(1, keepdim=True)
    r = (X - mu).square().mean(1, keepdim=True).add(eps).rsqrt()
    xh = (X - mu) * r
    k = (max(c, 2) - 1).bit_length() + 8
    xh_err = k * E * (r * (X.abs() + X.abs().mean(1, keepdim=True)) + 2 * xh.abs())
    u, uw, t, tw = U[dtype], U[wtype], TINY[dtype], TINY[wtype]
    want = dict(y=xh * W + Bv, mean=mu[:, 0], rstd=r[:, 0])
    tol = dict(y=u * want["y"].abs() + xh_err * W.abs() + 2 * E * (W * xh).abs() + t,
               mean=k * E * X.abs().mean(1), rstd=k * E * (r[:, 0] + (r * r * xh_err.mean(1, keepdim=True))[:, 0] + r[:, 0]))
    v = G * W
    m1, m2 = v.mean(1, keepdim=True), (v * xh).mean(1, keepdim=True)
    want.update(dx=r * (v - m1 - xh * m2), dw=(G * xh).sum(0), db=G.sum(0))
    va = v.abs()
    m2_err = (va * xh_err).mean(1, keepdim=True) + k * E * (va * xh.abs()).mean(1, keepdim=True)
    tol.update(dx=u * want["dx"].abs() + t + r * (4 * k * E * (va + va.mean(1, keepdim=True) + (xh * m2).abs())
                                                  + xh_err * m2.abs() + xh.abs() * m2_err),
               dw=uw * want["dw"].abs() + tw + (G.abs() * xh_err).sum(0) + (n + 40) * E * (G * xh).abs().sum(0),
               db=uw * want["db"].abs() + tw + (n + 40) * E * G.abs().sum(0))
    got = dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)
    for name in want:
        off = (got[name].double() - want[name]).abs() - 1.25 * tol[name]
        assert not torch.isnan(off).any(), name
        assert off.max().item() <= 0, (name, off.max().item())


@pytest.mark.parametrize("dtype,wtype", [("f32", "f32"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (1, 8192), (5, 7), (33, 64), (130, 255), (67, 771), (300, 1024), (9, 1025),
                                       (40, 2048), (21, 2049), (17, 4096), (10, 8191), (5000, 96)])
def test_values_and_gradients(ddm, dtype, wtype, rows, cols):
    check(ddm, *make(rows, cols, dtype, wtype, seed=cols), dtype, wtype, eps=1e-6 if cols > 2 else 1e-2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_weight_and_bias(ddm, dtype):
    x, w, b, dy = make(50, 320, dtype, "f32")
    check(ddm, x, None, None, dy, dtype, "f32")
    check(ddm, x, w, None, dy, dtype, "f32")
    check(ddm, x, None, b, dy, dtype, "f32")


def test_mean_far_larger_than_spread(ddm):
    """The variance is taken about the mean, not from the sum of squares."""
    x, w, b, dy = make(64, 500, "f32", "f32", seed=3)
    check(ddm, x + 1000, w, b, dy, "f32", "f32")


def test_constant_rows(ddm):
    x = torch.full((4, 300), 2.5, device="cuda")
    y, mean, rstd = ddm.layer_norm_forward(x, eps=1e-4)
    assert (y == 0).all() and (mean == 2.5).all() and torch.allclose(rstd, torch.full_like(rstd, 100.0))


def test_nan_stays_in_its_row(ddm):
    x, w, b, dy = make(10, 600, "bf16", "f32", seed=4)
    y0, _, _ = ddm.layer_norm_forward(x, w, b)
    x[3, 5] = float("nan")
    x[7, 599] = float("inf")
    y, mean, _ = ddm.layer_norm_forward(x, w, b)
    keep = [i for i in range(10) if i not in (3, 7)]
    assert torch.equal(y[keep], y0[keep]) and torch.isnan(y[3]).all() and torch.isnan(mean[3]) and torch.isnan(y[7]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_row_stride_and_odd_addresses(ddm, dtype):
    base, w, b, _ = make(40, 700, dtype, "f32", seed=5)
    x = base[:, 3:336]                                   # 333 columns, rows 700 apart, first element off a 16-byte boundary
    dy = torch.randn(40 * 333 + 1, device="cuda").to(DT[dtype])[1:].view(40, 333)
    w, b = w[1:334], b[1:334]
    y, mean, rstd = ddm.layer_norm_forward(x, w, b)
    y2, mean2, rstd2 = ddm.layer_norm_forward(x.contiguous(), w.clone(), b.clone())
    assert torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    for s, t in zip(ddm.layer_norm_backward(dy, x, w, mean, rstd),
                    ddm.layer_norm_backward(dy.clone(), x.contiguous(), w.clone(), mean, rstd)):
        assert torch.equal(s, t)


def test_no_rows_and_leading_dimensions(ddm):
    w = torch.ones(64, device="cuda")
    y, mean, rstd = ddm.layer_norm_forward(torch.zeros(0, 64, device="cuda"), w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = ddm.layer_norm_backward(y, y, w, mean, rstd)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    x = torch.randn(2, 3, 64, device="cuda")
    y, mean, _ = ddm.layer_norm_forward(x, w)
    assert y.shape == x.shape and mean.shape == (2, 3)


def test_parts_and_repeats(ddm):
    x, w, b, dy = make(3000, 384, "bf16", "f32", seed=6)
    _, mean, rstd = ddm.layer_norm_forward(x, w, b)
    full = ddm.layer_norm_backward(dy, x, w, mean, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = ddm.layer_norm_backward(dy, x, w, mean, rstd)
    s.synchronize()
    for p, q in zip(full, again):
        assert torch.equal(p, q)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        got = ddm.layer_norm_backward(dy, x, w, mean, rstd, need_dx=need[0], need_dweight=need[1], need_dbias=need[2])
        for g, f, n in zip(got, full, need):
            assert torch.equal(g, f) if n else g is None


def test_graph_replays(ddm):
    x, w, b, dy = make(500, 1024, "bf16", "f32", seed=7)

    def step():
        y, mean, rstd = ddm.layer_norm_forward(x, w, b)
        return (y,) + ddm.layer_norm_backward(dy, x, w, mean, rstd)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)


def test_autograd_and_differences(ddm):
    """Differences in 64 bits of the definition agree with autograd's float32 gradient to its rounding."""
    x, w, b, dy = make(6, 40, "f32", "f32", seed=8)
    t = [v.clone().requires_grad_() for v in (x, w, b)]
    (ddm.layer_norm(*t, eps=1e-5) * dy).sum().backward()

    def f(x, w, b):
        x = x - x.mean(1, keepdim=True)
        return ((x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w + b) * dy.double()).sum()

    base = [v.double() for v in (x, w, b)]
    for i in range(3):
        d = torch.randn_like(base[i])
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + 1e-4 * d, base[i] - 1e-4 * d
        diff = (f(*up) - f(*down)) / 2e-4
        want = (t[i].grad.double() * d).sum()
        assert abs(diff - want) <= 1e-4 * (1 + t[i].grad.double().norm() * d.norm())


def test_refusals(ddm):
    x, w, b, dy = make(4, 64, "bf16", "f32")
    f = ddm.layer_norm_forward
    with pytest.raises(TypeError):
        f(x.cpu(), w, b)
    with pytest.raises(TypeError):
        f(x.double(), w, b)
    with pytest.raises(TypeError):
        f(x, w.half(), b.half())                         # neither float32 nor x's type
    with pytest.raises(TypeError):
        f(x, w, b.bfloat16())
    with pytest.raises(ValueError):
        f(x, w[:63], b)
    with pytest.raises(ValueError):
        f(x.t(), None, None)
    with pytest.raises(ddm.DDMError) as e:
        f(torch.zeros(1, 8193, device="cuda"))
    assert e.value.status == -4
    for eps in (-1.0, float("inf"), float("nan")):
        with pytest.raises(ddm.DDMError) as e:
            f(x, w, b, eps=eps)
        assert e.value.status == -1
    _, mean, rstd = f(x, w, b)
    with pytest.raises(ValueError):
        ddm.layer_norm_backward(dy.t(), x, w, mean, rstd)
    with pytest.raises(TypeError):
        ddm.layer_norm_backward(dy.float(), x, w, mean, rstd)
