"""NaN in a query or a key shows in what depends on it, never as the -inf of a query that sees no key, and nowhere else."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import ddm, make, run  # noqa: E402,F401  (ddm is a fixture)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,row", [(((70, 200), (70, 200)), 130), (((1, 2), (2000, 3000)), 2)])
def test_query_of_nan(ddm, dtype, lens, row):
    x = make(dtype, 4, 2, 64, *lens, seed=32)
    want = run(ddm, x, True, 0.125)
    x["q"][row, 1, 3] = float("nan")
    got = run(ddm, x, True, 0.125)
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
def test_key_of_nan(ddm, dtype, lens):
    """Queries that see the key have NaN, those that do not keep their values, and those that see none have -inf."""
    x = make(dtype, 4, 2, 64, *lens, seed=33)
    want = run(ddm, x, True, 0.125)
    m, n = lens[0][1], lens[1][1]
    q0, k0 = lens[0][0], lens[1][0]
    key = n - 2                                          # the last query of the sequence but one sees it as its last key
    x["k"][k0 + key, 1, 7] = float("nan")
    got = run(ddm, x, True, 0.125)
    sees = torch.zeros(sum(lens[0]), 4, dtype=torch.bool, device="cuda")
    sees[q0 + m - 2:q0 + m, 2:] = True
    assert torch.equal(torch.isnan(got["lse"]), sees)
    assert torch.isnan(got["out"][sees]).all() and torch.isnan(got["dq"][sees]).all()
    for name in ("out", "lse"):
        assert torch.equal(got[name][~sees], want[name][~sees]), name
    assert (got["lse"][-lens[0][2]:] == -math.inf).all() and (got["out"][-lens[0][2]:] == 0).all()
    assert torch.isnan(got["dv"][k0:k0 + n - 1, 1]).all()
