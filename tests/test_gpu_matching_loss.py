"""The matching loss and its gradient against the definition in 64 bits.

Tolerances per element: scores of unit-norm rows divided by the temperature t carry e = (d + 4 + 4 max|z|) 2^-24 of absolute error
(d times the largest |a_i| |b_j| where rows are scaled) from 32-bit products and exponents, which the losses and the lse take over twice and every exponential relatively; sums over
n columns add (n / 8 + 16) 2^-24 relatively (partial sums of lanes and tiles). Off the diagonal the gradient by a score is rounded once to the inputs' type
(u = 2^-8 bfloat16, 2^-11 float16, and 2^-25 of the largest dloss at least in float16) before it multiplies the other side's
rows; da and db are rounded once.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
E = 2.0 ** -24
ALL = ("loss", "lse_a", "lse_b", "da", "db")


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


def cu_of(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def make(dtype, d, lens, seed=0, pad=0, noise=1.2, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    p = sum(lens) + 2 * pad
    a = torch.nn.functional.normalize(torch.randn(p, d, generator=g, device="cuda"), dim=1)
    b = torch.nn.functional.normalize(a + noise * torch.randn(p, d, generator=g, device="cuda") / d ** 0.5, dim=1)
    return dict(a=a.to(DT[dtype]), b=b.to(DT[dtype]), cu=cu_of(lens, pad),
                g=(torch.rand(p, generator=g, device="cuda") - 0.2) * scale)


def run(ddm, x, t=0.07):
    loss, la, lb = ddm.matching_loss_forward(x["a"], x["b"], x["cu"], temperature=t)
    da, db = ddm.matching_loss_backward(x["g"], x["a"], x["b"], la, lb, x["cu"], temperature=t)
    return dict(loss=loss, lse_a=la, lse_b=lb, da=da, db=db)


def check(got, x, dtype, t=0.07, norms=1.0):
    u = U[dtype]
    cu = x["cu"].tolist()
    d = x["a"].shape[1]
    for lo, hi in zip(cu, cu[1:]):
        n = hi - lo
        if n == 0:
            continue
        a, b, g = (x[k][lo:hi].double() for k in ("a", "b", "g"))
        z = a @ b.T / t
        la, lb = torch.logsumexp(z, 1), torch.logsumexp(z, 0)
        e = (d * norms + 4 + 4 * float(z.abs().max())) * E
        s = 2 * e + (n / 8 + 16) * E
        pa, pb = torch.exp(z - la[:, None]) * g[:, None] / 2, torch.exp(z - lb[None, :]) * g[None, :] / 2
        dz = pa + pb - torch.diag(g)
        eye = torch.eye(n, dtype=torch.float64, device="cuda")
        dz_err = (2 * s + 4 * E) * (pa.abs() + pb.abs() + torch.diag(g.abs())) + u * dz.abs() * (1 - eye)
        if dtype == "f16":
            dz_err += 2.0 ** -25 * 2 * g.abs().max()
        want = dict(loss=(la + lb) / 2 - z.diagonal(), lse_a=la, lse_b=lb, da=dz @ b / t, db=dz.T @ a / t)
        tol = dict(loss=torch.full_like(la, 2 * s) + 4 * E, lse_a=s + 4 * E * la.abs(), lse_b=s + 4 * E * lb.abs(),
                   da=(dz_err + (n / 8 + 16) * E * dz.abs()) @ b.abs() / t, db=(dz_err + (n / 8 + 16) * E * dz.abs()).T @ a.abs() / t)
        for k in ("da", "db"):
            tol[k] += (u or E) * want[k].abs() + (2.0 ** -25 if dtype == "f16" else 0)
        for k in ALL:
            off = (got[k][lo:hi].double() - want[k]).abs() - 1.25 * tol[k]
            assert not torch.isnan(off).any(), k
            assert off.max().item() <= 0, (k, off.max().item())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [1, 3, 8, 16, 24, 31, 33, 64, 100, 128])
@pytest.mark.parametrize("lens", [(1,), (2, 1, 0, 65), (300, 129), (1000,)])
def test_values_and_gradients(ddm, dtype, d, lens):
    x = make(dtype, d, lens, seed=d)
    check(run(ddm, x), x, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_larger_sets(ddm, dtype):
    """Sizes at which the columns are cut into several pieces, and at which they are not."""
    for lens in ((4000, 2500, 77), (128,) * 520):
        x = make(dtype, 24, lens, seed=1)
        check(run(ddm, x), x, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [16, 33, 64, 128])
@pytest.mark.parametrize("lens", [(4200,), (1025, 0, 513, 1, 3000, 128, 127)])
def test_one_pass(ddm, dtype, d, lens):
    """From 4096 matches on one exponential of a score serves both directions."""
    x = make(dtype, d, lens, seed=11)
    check(run(ddm, x), x, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_one_and_two_passes_together(ddm, dtype):
    """Scores of some sets lie within 32 and those of others do not."""
    lens = (2000, 1500, 1, 0, 700, 300)
    x = make(dtype, 24, lens, seed=12, noise=0.8)
    for i in (1, 4):
        lo, hi = sum(lens[:i]), sum(lens[:i + 1])
        x["a"][lo:hi] *= 3
        x["b"][lo:hi] *= 3
    check(run(ddm, x), x, dtype, norms=9.0)


def test_a_set_too_long_for_one_pass(ddm):
    x = make("f16", 16, (32769, 500), seed=13, scale=16.0)
    check(run(ddm, x), x, "f16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_clear_matches(ddm, dtype):
    x = make(dtype, 64, (4500, 1), seed=14, noise=0.05)
    got = run(ddm, x)
    check(got, x, dtype)
    assert got["loss"][-1].item() == 0


def test_one_pass_has_the_same_bits_in_graph_replays_and_between_other_rows(ddm):
    x = make("bf16", 24, (3000, 2500), seed=15, pad=9)
    want = run(ddm, x)
    for n in ("a", "b", "g"):
        x[n][:9], x[n][-9:] = float("nan"), float("inf")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ddm, x)
    for _ in range(3):
        for t in got.values():
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for n in ALL:
            assert torch.equal(got[n][9:-9], want[n][9:-9])
            assert (got[n][:9] == 0).all() and (got[n][-9:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_clear_matches(ddm, dtype):
    """Nearly equal rows: the loss is the logarithm of a sum next to 1 and keeps its absolute precision."""
    x = make(dtype, 64, (500,), seed=2, noise=0.05)
    check(run(ddm, x), x, dtype)


def test_small_upstream_gradients_in_half_precision(ddm):
    x = make("f16", 24, (700, 300), seed=3, scale=2.0 ** -9)
    check(run(ddm, x), x, "f16")


@pytest.mark.parametrize("t", [0.01, 1.0, 50.0])
def test_temperatures(ddm, t):
    x = make("f32", 24, (200, 90), seed=4)
    check(run(ddm, x, t), x, "f32", t)


@pytest.mark.parametrize("dtype,d", [("bf16", 24), ("f32", 33)])
def test_rows_outside_every_set(ddm, dtype, d):
    pad = 7
    x = make(dtype, d, (60, 0, 100), seed=5, pad=pad)
    want = run(ddm, x)
    for n in ("a", "b", "g"):
        x[n][:pad], x[n][-pad:] = float("nan"), float("inf")
    got = run(ddm, x)
    for n in ALL:
        assert torch.equal(got[n][pad:-pad], want[n][pad:-pad])
        assert (got[n][:pad] == 0).all() and (got[n][-pad:] == 0).all()
    check({k: v for k, v in got.items()}, x, dtype)


def test_odd_addresses(ddm):
    x = make("bf16", 24, (150,), seed=6)
    want = run(ddm, x)
    odd = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    got = run(ddm, dict(x, a=odd(x["a"]), b=odd(x["b"])))
    for n in ALL:
        assert torch.equal(got[n], want[n])


def test_empty_and_single(ddm):
    z = torch.zeros(0, 24, device="cuda")
    loss, la, lb = ddm.matching_loss_forward(z, z)
    assert loss.shape == (0,)
    da, db = ddm.matching_loss_backward(loss, z, z, la, lb)
    assert da.shape == (0, 24)
    x = make("f32", 24, (1,), seed=7)
    got = run(ddm, x)
    assert got["loss"].item() == 0 and got["da"].abs().max().item() <= 1e-5


def test_bad_boundaries_stay_inside(ddm):
    x = make("bf16", 24, (50, 70), seed=8)
    want = run(ddm, x)
    got = run(ddm, dict(x, cu=torch.tensor([-3, 50, 10 ** 6], dtype=torch.int32, device="cuda")))
    for n in ALL:
        assert torch.equal(got[n], want[n])


def test_same_bits_on_a_side_stream_and_in_graph_replays(ddm):
    x = make("f16", 24, (900, 300), seed=9)
    want = run(ddm, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(ddm, x)
    s.synchronize()
    for n in ALL:
        assert torch.equal(got[n], want[n])
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ddm, x)
    for _ in range(3):
        for t in got.values():
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for n in ALL:
            assert torch.equal(got[n], want[n])


def test_autograd_and_differences(ddm):
    x = make("f32", 24, (40, 25), seed=10)
    a, b = (x[k].clone().requires_grad_() for k in ("a", "b"))
    (ddm.matching_loss(a, b, x["cu"]) * x["g"]).sum().backward()
    cu = x["cu"].tolist()

    def f(a, b):
        total = 0.0
        for lo, hi in zip(cu, cu[1:]):
            z = a[lo:hi] @ b[lo:hi].T / 0.07
            total = total + (((torch.logsumexp(z, 1) + torch.logsumexp(z, 0)) / 2 - z.diagonal()) * x["g"][lo:hi].double()).sum()
        return total

    for i, t in enumerate((a, b)):
        w = torch.randn(t.shape, dtype=torch.float64, device="cuda")
        up, down = [a.detach().double(), b.detach().double()], [a.detach().double(), b.detach().double()]
        up[i] = up[i] + 1e-5 * w
        down[i] = down[i] - 1e-5 * w
        diff = (f(*up) - f(*down)) / 2e-5
        want = (t.grad.double() * w).sum()
        assert abs(diff - want) <= 1e-4 * t.grad.double().norm() * w.norm()


def test_refusals(ddm):
    x = make("bf16", 24, (8,))
    a, b = x["a"], x["b"]
    f = ddm.matching_loss_forward
    with pytest.raises(TypeError):
        f(a.cpu(), b.cpu())
    with pytest.raises(TypeError):
        f(a, b.float())
    with pytest.raises(ValueError):
        f(a, b[:7])
    with pytest.raises(ValueError):
        f(a[:, :12], b[:, :12])                          # rows not contiguous
    with pytest.raises(ValueError):
        f(a[0], b[0])
    with pytest.raises(TypeError):
        f(a, b, x["cu"].long())
    with pytest.raises(ValueError):
        f(a, b, x["cu"][:1])
    for t in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ddm.DDMError) as e:
            f(a, b, temperature=t)
        assert e.value.status == -1
    wide = torch.zeros(4, 129, device="cuda")
    with pytest.raises(ddm.DDMError) as e:
        f(wide, wide)
    assert e.value.status == -4
    loss, la, lb = f(a, b)
    with pytest.raises(TypeError):
        ddm.matching_loss_backward(loss.half(), a, b, la, lb)
    with pytest.raises(ValueError):
        ddm.matching_loss_backward(loss[:7], a, b, la, lb)
