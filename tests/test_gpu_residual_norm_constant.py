"""Gradients of rows (or branches) that are one large value throughout: the mean is exact, the norm is zero, 1 / deviation is eps ** -1/2,
and dx = rstd (u - mean(u)) + ds. The mean times 1 / deviation is beyond 32 bits, in widths that fill the columns that a wave holds and in
others, whose missing columns count for nothing.

Tolerance: with E = 2^-24 and u the type's unit roundoff, a mean of C columns is a tree of log2 C + 8 roundings of the absolute terms;
their difference, 1 / deviation (4 roundings), its product and ds add 8 E of what they come to; then one rounding to the type."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
EPS, BIG = 1e-20, 2.0 ** 100


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


def through_norm(u):
    """rstd (u - mean(u)) in 64 bits, and its error."""
    u, rstd = u.double(), EPS ** -0.5
    k = u.shape[1].bit_length() + 8
    m = u.mean(1, keepdim=True)
    return rstd * (u - m), rstd * E * (k * u.abs().mean(1, keepdim=True) + 8 * (u.abs() + m.abs()))


def agrees(got, want, err):
    assert torch.isfinite(got).all()
    assert ((got.double() - want).abs() <= err + (U[got.dtype] + 8 * E) * want.abs()).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [1, 3, 64, 300, 1000, 1024, 1285, 2500, 4096, 5000, 8192])
def test_rows_of_one_large_value(ddm, dtype, cols):
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    x = torch.full((5, cols), BIG, device="cuda", dtype=dtype)
    zero = torch.zeros_like(x)
    dy, ds = (torch.randn(5, cols, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    s, y, stats = ddm.residual_norm_forward(x, zero, w, eps=EPS)
    assert torch.equal(s, x) and (y == 0).all() and (stats[0] == BIG).all()
    dx, dbranch, dw, db = ddm.residual_norm_backward(dy, ds, x, zero, stats, w)[:4]
    want, err = through_norm(dy.float() * w)
    want, err = want + ds.double(), err + 2 * E * EPS ** -0.5 * (dy.double() * w).abs()
    agrees(dx, want, err)
    agrees(dbranch, want, err)
    assert (dw == 0).all() and torch.isfinite(db).all()
    # the same in the branch, whose gradient by the sum is ds
    s, y, stats = ddm.residual_norm_forward(zero, x, w, branch_norm=True, eps=EPS)
    assert (s == 0).all() and (stats[2] == BIG).all()
    dx, dbranch, _, _, _, _, dbw, dbb = ddm.residual_norm_backward(None, ds, zero, x, stats, w, branch_norm=True)
    assert torch.equal(dx, ds) and (dbw == 0).all() and torch.isfinite(dbb).all()
    agrees(dbranch, *through_norm(ds))
