"""The residual norm against its definition in 64 bits.

Tolerances per element: u, the unit roundoff of an output's type (2^-8 bfloat16, 2^-11 float16, 2^-24 float32), of its value; before
that all is 32-bit with E = 2^-24. A sum over C columns is a tree: k = log2 C + 8 roundings of its absolute terms; one over N rows
has up to N + 40. The exponential of the gate g is off by (|g| + 2) 2 E of its value and the reciprocal by 2 E, which leaves
sigmoid(g) = o off by o (1 - o) (|g| + 2) 2 E + 4 E o. Errors run on through the formulas to first order; the factor 1.25 is for the
second.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
E = 2.0 ** -24
NAMES = ("dx", "dbranch", "dweight", "dbias", "dscale", "dgate", "dbranch_weight", "dbranch_bias")


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


def make(rows, cols, dtype, wtype, scale=True, gate=True, branch_norm=True, weight=True, bias=True, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, br, dy, ds = (t.to(DT[dtype]) for t in (r(rows, cols) * r(cols).mul(0.5).exp() + r(cols), r(rows, cols) + 0.3 * r(cols),
                                               r(rows, cols), r(rows, cols)))
    p = dict(weight=1 + 0.2 * r(cols) if weight else None, bias=0.2 * r(cols) if bias else None,
             scale=0.5 + 0.2 * r(cols) if scale else None, branch_weight=1 + 0.2 * r(cols) if branch_norm else None,
             branch_bias=0.2 * r(cols) if branch_norm else None)
    p = {n: None if t is None else t.to(DT[wtype]) for n, t in p.items()}
    p.update(gate=(2 * r(rows, cols)).to(DT[dtype]) if gate else None, branch_norm=branch_norm)
    return x, br, dy, ds, p


def normed(z, z_err, rms, eps, k):
    """norm(z), its error, 1 / deviation, its relative error, mean and its error."""
    mu = torch.zeros_like(z[:, :1]) if rms else z.mean(1, keepdim=True)
    mu_err = torch.zeros_like(mu) if rms else z_err.mean(1, keepdim=True) + k * E * z.abs().mean(1, keepdim=True)
    r = (z - mu).square().mean(1, keepdim=True).add(eps).rsqrt()
    h = (z - mu) * r
    first = r * (z_err + mu_err) + E * (r * (z.abs() + mu.abs()) + 2 * h.abs())
    rel = (h.abs() * first).mean(1, keepdim=True) + (k + 4) * E
    return h, first + h.abs() * rel, r, rel, mu, mu_err


def back(v, v_err, h, h_err, r, rel, rms, k):
    """Gradient through norm, and its error."""
    m1 = torch.zeros_like(r) if rms else v.mean(1, keepdim=True)
    m2 = (v * h).mean(1, keepdim=True)
    m1_err = torch.zeros_like(r) if rms else v_err.mean(1, keepdim=True) + k * E * v.abs().mean(1, keepdim=True)
    m2_err = (v_err * h.abs() + v.abs() * h_err).mean(1, keepdim=True) + k * E * (v * h).abs().mean(1, keepdim=True)
    out = r * (v - m1 - h * m2)
    err = r * (v_err + m1_err + h_err * m2.abs() + h.abs() * m2_err + 3 * E * (v.abs() + m1.abs() + (h * m2).abs())) + rel * out.abs()
    return out, err


def expected(x, br, dy, ds, p, rms, eps, dtype, wtype):
    n, c = x.shape
    k = (max(c, 2) - 1).bit_length() + 8
    x, br, dy, ds = (t.double() for t in (x, br, dy, ds))
    one, nil = torch.ones(c, dtype=torch.float64, device="cuda"), torch.zeros(c, dtype=torch.float64, device="cuda")
    w, b, sc, bw, bb = ((p[m].double() if p[m] is not None else d) for m, d in (("weight", one), ("bias", nil), ("scale", one),
                                                                               ("branch_weight", one), ("branch_bias", nil)))
    want, tol = {}, {}
    t, t_err, stats, stats_err = br, torch.zeros_like(br), [], []
    if p["branch_norm"]:
        bh, bh_err, bR, b_rel, bmu, bmu_err = normed(br, torch.zeros_like(br), rms, eps, k)
        t = bh * bw + bb
        t_err = bh_err * bw.abs() + 2 * E * ((bh * bw).abs() + t.abs())
        stats, stats_err = [bmu, bR], [bmu_err, b_rel * bR]
    o, o_err = torch.ones_like(t), torch.zeros_like(t)
    if p["gate"] is not None:
        g = p["gate"].double()
        o = torch.sigmoid(g)
        o_err = o * (1 - o) * (g.abs() + 2) * 2 * E + 4 * E * o
    part = t * o
    part_err = t_err * o + t.abs() * o_err + E * part.abs()
    s = x + sc * part
    s_err = sc.abs() * part_err + E * ((sc * part).abs() + s.abs())
    h, h_err, R, rel, mu, mu_err = normed(s, s_err, rms, eps, k)
    u, tiny, uw, tw = U[dtype], TINY[dtype], U[wtype], TINY[wtype]
    want["s"], tol["s"] = s, u * s.abs() + tiny + s_err
    want["y"] = h * w + b
    tol["y"] = u * want["y"].abs() + tiny + h_err * w.abs() + 2 * E * (h * w).abs() + E * want["y"].abs()
    want["stats"] = torch.stack([v[:, 0] for v in [mu, R] + stats])
    tol["stats"] = torch.stack([v[:, 0] for v in [mu_err + E * mu.abs(), rel * R] + stats_err]) + 2 * E * want["stats"].abs()
    rows = (n + 40) * E

    def summed(name, a, a_err, d, d_err):
        want[name] = (a * d).sum(0)
        tol[name] = uw * want[name].abs() + tw + (a_err * d.abs() + a.abs() * d_err).sum(0) + rows * (a * d).abs().sum(0)

    zero = torch.zeros_like(x)
    summed("dweight", dy, zero, h, h_err)
    summed("dbias", dy, zero, torch.ones_like(x), zero)
    v = dy * w
    z, z_err = back(v, E * v.abs(), h, h_err, R, rel, rms, k)
    dx, dx_err = ds + z, z_err + E * (ds + z).abs()
    want["dx"], tol["dx"] = dx, u * dx.abs() + tiny + dx_err
    summed("dscale", dx, dx_err, part, part_err)
    v = dx * sc
    v_err = dx_err * sc.abs() + E * v.abs()
    if p["gate"] is not None:
        slope = o * (1 - o)
        want["dgate"] = v * t * slope
        tol["dgate"] = u * want["dgate"].abs() + tiny + v_err * (t * slope).abs() + v.abs() * (
            t_err * slope + t.abs() * (o_err * (1 + o) + 4 * E * slope + 2 * E * o))
        v_err = v_err * o + v.abs() * o_err + E * (v * o).abs()
        v = v * o
    if p["branch_norm"]:
        summed("dbranch_weight", v, v_err, bh, bh_err)
        summed("dbranch_bias", v, v_err, torch.ones_like(x), zero)
        v_err = v_err * bw.abs() + E * (v * bw).abs()
        v, v_err = back(v * bw, v_err, bh, bh_err, bR, b_rel, rms, k)
    want["dbranch"], tol["dbranch"] = v, u * v.abs() + tiny + v_err
    return want, tol


def run(ddm, x, br, dy, ds, p, rms, eps, wtype):
    f = {n: p[n] for n in ("scale", "gate", "branch_norm", "branch_weight", "branch_bias")}
    s, y, stats = ddm.residual_norm_forward(x, br, p["weight"], p["bias"], rms=rms, eps=eps, **f)
    needs = set(NAMES) - (set() if p["gate"] is not None else {"dgate"}) - (
        set() if p["branch_norm"] else {"dbranch_weight", "dbranch_bias"})
    grads = ddm.residual_norm_backward(dy, ds, x, br, stats, p["weight"], rms=rms, wtype=DT[wtype], needs=needs, **f)
    return dict(s=s, y=y, stats=stats, **{n: g for n, g in zip(NAMES, grads) if g is not None})


def check(ddm, args, dtype, wtype, rms=False, eps=1e-6):
    got = run(ddm, *args, rms, eps, wtype)
    want, tol = expected(*args, rms, eps, dtype, wtype)
    assert got.keys() == want.keys()
    for name in want:
        off = (got[name].double() - want[name]).abs() - 1.25 * tol[name]
        assert not torch.isnan(off).any(), name
        assert off.max().item() <= 0, (name, off.max().item())


@pytest.mark.parametrize("dtype,wtype", [("f32", "f32"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (1, 8192), (5, 7), (33, 64), (130, 255), (67, 771), (300, 1024), (9, 1025),
                                       (40, 2048), (21, 2049), (17, 4096), (6, 4097), (10, 8191), (3000, 96)])
def test_values_and_gradients(ddm, dtype, wtype, rows, cols):
    check(ddm, make(rows, cols, dtype, wtype, seed=cols), dtype, wtype, rms=cols % 2 == 0, eps=1e-6 if cols > 2 else 1e-2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("parts", [dict(scale=False, gate=False, branch_norm=False), dict(gate=False, branch_norm=False),
                                   dict(scale=False, branch_norm=False), dict(scale=False, gate=False),
                                   dict(scale=False, gate=False, branch_norm=False, weight=False, bias=False),
                                   dict(weight=False), dict(bias=False)])
def test_parts_that_are_not_there(ddm, dtype, rms, parts):
    check(ddm, make(50, 330, dtype, "f32", seed=1, **parts), dtype, "f32", rms=rms)


def test_gate_far_open_and_shut(ddm):
    args = make(20, 200, "f32", "f32", seed=2)
    args[-1]["gate"] = torch.tensor([-1e30, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 1e30], device="cuda").repeat(20, 25)
    got = run(ddm, *args, False, 1e-6, "f32")
    assert all(torch.isfinite(t).all() for t in got.values())
    x, br, _, _, p = args
    assert torch.equal(got["s"][:, 0], x[:, 0]) and (got["dgate"][:, [0, 7]] == 0).all()


def test_constant_rows(ddm):
    x = torch.full((4, 300), 2.0, device="cuda")
    s, y, stats = ddm.residual_norm_forward(x, torch.full_like(x, 0.5), eps=1e-4)
    assert (s == 2.5).all() and (y == 0).all() and (stats[0] == 2.5).all()
    s, y, stats = ddm.residual_norm_forward(x, torch.full_like(x, 0.5), branch_norm=True, eps=1e-4)
    assert (s == 2.0).all() and (stats[2] == 0.5).all()


def test_nan_stays_in_its_row(ddm):
    x, br, dy, ds, p = make(10, 600, "bf16", "f32", seed=4)
    clean = run(ddm, x, br, dy, ds, p, False, 1e-6, "f32")
    x, br = x.clone(), br.clone()
    x[3, 5], br[7, 599] = float("nan"), float("inf")
    got = run(ddm, x, br, dy, ds, p, False, 1e-6, "f32")
    keep = [i for i in range(10) if i not in (3, 7)]
    for n in ("s", "y", "dx", "dbranch", "dgate"):
        assert torch.equal(got[n][keep], clean[n][keep]), n
    assert torch.isnan(got["y"][[3, 7]]).all() and torch.isnan(got["dweight"]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_row_strides_and_odd_addresses(ddm, dtype):
    x0, b0, dy, ds, p = make(40, 333, dtype, "f32", seed=5)
    wide = torch.empty(40, 1003, device="cuda", dtype=DT[dtype])
    views = [wide[:, i:i + 333] for i in (1, 334, 667)]
    for v, t in zip(views, (x0, b0, p["gate"])):
        v.copy_(t)
    want = run(ddm, x0, b0, dy, ds, p, False, 1e-6, "f32")
    odd = torch.empty(334 * 5 + 1, device="cuda")[1:]
    q = dict(p, gate=views[2])
    for i, n in enumerate(("weight", "bias", "scale", "branch_weight", "branch_bias")):
        q[n] = odd[334 * i:334 * i + 333].copy_(p[n])
    got = run(ddm, views[0], views[1], dy, ds, q, False, 1e-6, "f32")
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_no_rows_and_leading_dimensions(ddm):
    w = torch.ones(64, device="cuda")
    e = torch.zeros(0, 64, device="cuda")
    s, y, stats = ddm.residual_norm_forward(e, e, w, scale=w, branch_norm=True)
    assert s.shape == y.shape == (0, 64) and stats.shape == (4, 0)
    grads = ddm.residual_norm_backward(y, s, e, e, stats, w, scale=w, branch_norm=True)
    assert grads[0].shape == (0, 64) and all((g == 0).all() for g in grads if g is not None and g.dim() == 1)
    x = torch.randn(2, 3, 64, device="cuda")
    s, y, stats = ddm.residual_norm_forward(x, x, w)
    assert s.shape == y.shape == x.shape and stats.shape == (2, 2, 3) and torch.equal(s, 2 * x)


def test_parts_repeats_and_zeros(ddm):
    x, br, dy, ds, p = make(2000, 384, "bf16", "f32", seed=6)
    f = {n: p[n] for n in ("scale", "gate", "branch_norm", "branch_weight", "branch_bias")}
    _, _, stats = ddm.residual_norm_forward(x, br, p["weight"], p["bias"], **f)
    call = lambda dy=dy, ds=ds, **kw: ddm.residual_norm_backward(dy, ds, x, br, stats, p["weight"], **f, **kw)  # noqa: E731
    full = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = call()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(full, again))
    for needs in ({"dx"}, {"dbranch"}, {"dgate", "dscale"}, {"dweight", "dbranch_bias"}, set(NAMES), set()):
        for n, g, w in zip(NAMES, call(needs=needs), full):
            assert torch.equal(g, w) if n in needs else g is None
    zero = torch.zeros_like(x)
    for kw, same in ((dict(dy=None), dict(dy=zero)), (dict(ds=None), dict(ds=zero))):
        assert all(torch.equal(a, b) for a, b in zip(call(**kw), call(**same)))


def test_graph_replays(ddm):
    args = make(500, 1024, "bf16", "f32", seed=7)
    want = run(ddm, *args, False, 1e-6, "f32")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ddm, *args, False, 1e-6, "f32")
    for _ in range(3):
        for t in got.values():
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_autograd_and_differences(ddm):
    """Differences in 64 bits of the definition agree with autograd's float32 gradient to its rounding."""
    x, br, dy, ds, p = make(6, 40, "f32", "f32", seed=8)
    names = ("weight", "bias", "scale", "gate", "branch_weight", "branch_bias")
    t = [v.clone().requires_grad_() for v in (x, br, *(p[n] for n in names))]
    s, y = ddm.residual_norm(*t[:4], scale=t[4], gate=t[5], branch_norm=True, branch_weight=t[6], branch_bias=t[7], eps=1e-5)
    ((s * ds).sum() + (y * dy).sum()).backward()

    def norm(z):
        z = z - z.mean(1, keepdim=True)
        return z * (z.square().mean(1, keepdim=True) + 1e-5).rsqrt()

    def f(x, br, w, b, sc, g, bw, bb):
        s = x + sc * torch.sigmoid(g) * (norm(br) * bw + bb)
        return (s * ds.double()).sum() + ((norm(s) * w + b) * dy.double()).sum()

    base = [v.detach().double() for v in t]
    for i in range(8):
        d = torch.randn_like(base[i])
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + 1e-4 * d, base[i] - 1e-4 * d
        diff = (f(*up) - f(*down)) / 2e-4
        assert abs(diff - (t[i].grad.double() * d).sum()) <= 1e-4 * (1 + t[i].grad.double().norm() * d.norm()), i
    for use in (0, 1):                                   # one output unused
        t = [v.clone().requires_grad_() for v in (x, br)]
        out = ddm.residual_norm(*t)[use]
        out.sum().backward()
        assert all(torch.isfinite(v.grad).all() for v in t)
        if use == 0:
            assert (t[0].grad == 1).all() and (t[1].grad == 1).all()


def test_refusals(ddm):
    x, br, dy, ds, p = make(4, 64, "bf16", "f32")
    f, w = ddm.residual_norm_forward, p["weight"]
    for bad in ((x.cpu(), br), (x.double(), br.double()), (x, br.float()), (x, br, w.half())):
        with pytest.raises((TypeError, ValueError)):
            f(*bad)
    for bad in (dict(gate=x.float()), dict(scale=w.bfloat16()), dict(branch_norm=True, branch_weight=w.bfloat16())):
        with pytest.raises(TypeError):
            f(x, br, w, **bad)
    for bad in (dict(gate=x[:3]), dict(scale=w[:63]), dict(branch_weight=w), dict(branch_bias=w)):
        with pytest.raises(ValueError):
            f(x, br, w, **bad)
    with pytest.raises(ValueError):
        f(x.t(), br.t())
    with pytest.raises(ValueError):
        f(x, br[:3])
    with pytest.raises(ddm.DDMError) as e:
        f(torch.zeros(1, 8193, device="cuda"), torch.zeros(1, 8193, device="cuda"))
    assert e.value.status == -4
    for eps in (-1.0, float("inf"), float("nan")):
        with pytest.raises(ddm.DDMError) as e:
            f(x, br, eps=eps)
        assert e.value.status == -1
    _, _, stats = f(x, br, w)
    b = ddm.residual_norm_backward
    with pytest.raises(ValueError):
        b(dy.t(), ds, x, br, stats, w)
    with pytest.raises(TypeError):
        b(dy.float(), ds, x, br, stats, w)
    with pytest.raises(ValueError):
        b(dy, ds, x, br, stats, w, branch_norm=True)
    for needs in ({"dgate"}, {"dbranch_weight"}, {"dz"}):
        with pytest.raises(ValueError):
            b(dy, ds, x, br, stats, w, needs=needs)
