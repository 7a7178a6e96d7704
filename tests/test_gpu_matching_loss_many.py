"""The matching loss in calls of very many matches, of which a few sets are checked; the other rows belong to no set."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_matching_loss import ALL, check, ddm, make, run  # noqa: E402,F401  (ddm is a fixture)

LENS = (3000, 1, 0, 1025, 129, 9000)


@pytest.mark.parametrize("rows", [(1 << 18) + 5, (1 << 19) + 5, (1 << 22) + 9])
def test_sets_among_many_rows(ddm, rows):
    pad = (rows - sum(LENS) + 1) // 2
    x = make("bf16", 24, LENS, seed=51, pad=pad)
    got = run(ddm, x)
    check(got, x, "bf16")
    for n in ALL:
        assert (got[n][:pad] == 0).all() and (got[n][-pad:] == 0).all(), n


def test_a_long_set_among_many_rows(ddm):
    x = make("f16", 16, (32768, 40), seed=52, pad=1 << 18, scale=16.0)
    check(run(ddm, x), x, "f16")
