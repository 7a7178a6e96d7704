"""NaN in a descriptor shows in the loss and the gradients of its set, never as a loss of 0, and nowhere else."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_matching_loss import ALL, ddm, make, run  # noqa: E402,F401  (ddm is a fixture)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("side", ["a", "b"])
@pytest.mark.parametrize("lens,scale", [((10,) * 250, 1.0), ((100, 30), 1.0), ((1000, 500), 1.0), ((2500, 2000, 300), 1.0),
                                        ((2500, 2000, 300), 3.0), ((1, 1, 1), 1.0)])
def test_nan_in_one_descriptor(ddm, dtype, side, lens, scale):
    """One NaN in a_r: lse_a_r and every lse_b of its set are NaN, so all losses and gradients of the set are; other sets keep
    their bits. Few and many pieces, one pass and (descriptors three times as long) two."""
    x = make(dtype, 24, lens, seed=31)
    x["a"], x["b"] = x["a"] * scale, x["b"] * scale
    want = run(ddm, x)
    lo = lens[0]
    hi = lo + lens[1]
    row = (lo + hi) // 2
    x[side][row, 5] = float("nan")
    got = run(ddm, x)
    for n in ALL:
        assert torch.equal(got[n][:lo], want[n][:lo]) and torch.equal(got[n][hi:], want[n][hi:]), n
    for n in ("loss", "da", "db", "lse_b" if side == "a" else "lse_a"):
        assert torch.isnan(got[n][lo:hi]).all(), n
    own = torch.isnan(got["lse_a" if side == "a" else "lse_b"][lo:hi])
    assert own[row - lo] and own.sum() == 1
