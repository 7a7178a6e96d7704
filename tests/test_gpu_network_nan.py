"""NaN inside a sequence or a set shows where the formulas carry it, and nowhere else: it neither becomes a loss of 0 nor the
-inf of a query that sees no key."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_attention as attention  # noqa: E402
import test_gpu_matching_loss as matching  # noqa: E402
from test_gpu_attention import ddm  # noqa: E402,F401  (a fixture)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("side", ["a", "b"])
@pytest.mark.parametrize("lens,scale", [((10,) * 250, 1.0), ((100, 30), 1.0), ((1000, 500), 1.0), ((2500, 2000, 300), 1.0),
                                        ((2500, 2000, 300), 3.0), ((1, 1, 1), 1.0)])
def test_matching_loss(ddm, dtype, side, lens, scale):
    """One NaN in a_r: lse_a_r and every lse_b of its set are NaN, so all losses and gradients of the set are; other sets keep
    their bits. Few and many pieces, one pass and (descriptors three times as long) two."""
    x = matching.make(dtype, 24, lens, seed=31)
    x["a"], x["b"] = x["a"] * scale, x["b"] * scale
    want = matching.run(ddm, x)
    lo = lens[0]
    hi = lo + lens[1]
    row = (lo + hi) // 2
    x[side][row, 5] = float("nan")
    got = matching.run(ddm, x)
    for n in matching.ALL:
        assert torch.equal(got[n][:lo], want[n][:lo]) and torch.equal(got[n][hi:], want[n][hi:]), n
    for n in ("loss", "da", "db", "lse_b" if side == "a" else "lse_a"):
        assert torch.isnan(got[n][lo:hi]).all(), n
    own = torch.isnan(got["lse_a" if side == "a" else "lse_b"][lo:hi])
    assert own[row - lo] and own.sum() == 1


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,row", [(((70, 200), (70, 200)), 130), (((1, 2), (2000, 3000)), 2)])
def test_attention_with_a_query_of_nan(ddm, dtype, lens, row):
    x = attention.make(dtype, 4, 2, 64, *lens, seed=32)
    want = attention.run(ddm, x, True, 0.125)
    x["q"][row, 1, 3] = float("nan")
    got = attention.run(ddm, x, True, 0.125)
    assert torch.isnan(got["lse"][row, 1]) and torch.isnan(got["out"][row, 1]).all() and torch.isnan(got["dq"][row, 1]).all()
    for n in ("out", "lse", "dq"):
        keep = torch.ones(got[n].shape[:2], dtype=torch.bool, device="cuda")
        keep[row, 1] = False
        assert torch.equal(got[n][keep], want[n][keep]), n
    first, seen = lens[1][0], lens[1][1] - lens[0][1] + row - lens[0][0] + 1     # keys that the row sees
    for n in ("dk", "dv"):
        assert torch.isnan(got[n][first:first + seen, 0]).all(), n
        assert torch.equal(got[n][:, 1], want[n][:, 1]) and torch.equal(got[n][:first], want[n][:first]), n


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens", [((70, 200, 5), (70, 200, 0)), ((3, 2, 1), (2000, 3000, 0))])
def test_attention_with_a_key_of_nan(ddm, dtype, lens):
    """Queries that see the key have NaN, those that do not keep their values, and those that see none have -inf."""
    x = attention.make(dtype, 4, 2, 64, *lens, seed=33)
    want = attention.run(ddm, x, True, 0.125)
    m, n = lens[0][1], lens[1][1]
    q0, k0 = lens[0][0], lens[1][0]
    key = n - 2                                          # the last query of the sequence but one sees it as its last key
    x["k"][k0 + key, 1, 7] = float("nan")
    got = attention.run(ddm, x, True, 0.125)
    sees = torch.zeros(sum(lens[0]), 4, dtype=torch.bool, device="cuda")
    sees[q0 + m - 2:q0 + m, 2:] = True
    assert torch.equal(torch.isnan(got["lse"]), sees)
    assert torch.isnan(got["out"][sees]).all() and torch.isnan(got["dq"][sees]).all()
    for name in ("out", "lse"):
        assert torch.equal(got[name][~sees], want[name][~sees]), name
    assert (got["lse"][-lens[0][2]:] == -math.inf).all() and (got["out"][-lens[0][2]:] == 0).all()
    assert torch.isnan(got["dv"][k0:k0 + n - 1, 1]).all()
