"""Many query heads on one key head, and sequences of very many rows."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import ALL, check, ddm, make, reference, run  # noqa: E402,F401  (ddm is a fixture)


def test_a_sequence_of_300000_tokens_of_128_heads(ddm):
    """38 million rows of one sequence: their numbers times the group's size pass 2^32. Without a mask a token's rows are a tile of
    their own and do not depend on others, so that calls for some of the tokens have the same bits; with causal masks only the
    last tokens see the few keys, and the call is that of those tokens alone."""
    n, keys, heads, dim = 300_000, 40, 128, 8
    x = make("bf16", heads, 1, dim, (n,), (keys,), seed=61)
    x["cu_q"] = x["cu_k"] = None
    some = lambda a, b: dict(x, q=x["q"][a:b], dout=x["dout"][a:b])  # noqa: E731
    got = run(ddm, x, False, 0.3)
    for a, b in ((0, 50), (131_000, 131_100), (262_100, 262_200), (n - 77, n)):
        want = run(ddm, some(a, b), False, 0.3)
        for m in ("out", "lse", "dq"):
            assert torch.equal(got[m][a:b], want[m]), (m, a)
    got = run(ddm, x, True, 0.3)
    want = run(ddm, some(n - keys, n), True, 0.3)
    assert (got["lse"][:n - keys] == -math.inf).all() and (got["out"][:n - keys] == 0).all() and (got["dq"][:n - keys] == 0).all()
    for m in ("out", "lse", "dq"):
        assert torch.equal(got[m][n - keys:], want[m]), m
    for m in ("dk", "dv"):                               # the same sums in other parts: 32-bit sums, and a rounding that they may move
        a, b = got[m].double(), want[m].double()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-3 * b.abs().max()).all(), m


def test_131072_packed_tokens_of_128_heads(ddm):
    """2^24 rows in 2048 sequences of the same 64 tokens: every one has the bits of the first, and its values."""
    x = make("bf16", 128, 1, 8, (64,), (64,), seed=62)
    val, tol = reference(x, True, 0.3, "bf16")
    many = {n: x[n].repeat(2048, 1, 1) for n in ("q", "k", "v", "dout")}
    cu = torch.arange(0, 131072 + 1, 64, dtype=torch.int32, device="cuda")
    got = run(ddm, dict(many, cu_q=cu, cu_k=cu), True, 0.3)
    for m in ALL:
        each = got[m].view(2048, 64, *got[m].shape[1:])
        assert (each == each[:1]).all(), m
        got[m] = each[0]
    check(got, val, tol, ALL)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads,kv", [(33, 1), (40, 1), (64, 1), (71, 1), (128, 1), (96, 2)])
@pytest.mark.parametrize("dim", [32, 64, 128])
def test_groups_larger_than_a_tile(ddm, dtype, causal, heads, kv, dim):
    """More query heads on a key head than the gradient's row tiles of 32 or 64 hold (a tile is then a whole part of one query's
    heads; of 71, a prime, one)."""
    x = make(dtype, heads, kv, dim, (30, 1, 17), (45, 3, 17), seed=63)
    check(run(ddm, x, causal, dim ** -0.5), *reference(x, causal, dim ** -0.5, dtype), ALL)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [((600,), (600,)), ((700, 90), (700, 600)), ((1, 1100), (40, 300)), ((900, 0, 330), (130, 70, 520))])
@pytest.mark.parametrize("heads,kv,dim", [(8, 1, 64), (24, 2, 128), (71, 1, 32)])
def test_rows_in_many_parts(ddm, dtype, causal, lens, heads, kv, dim):
    """Few key tiles and many rows: the gradient by keys and values cuts rows into up to eight parts and joins them, in
    sequences of as many parts, of fewer and of one."""
    x = make(dtype, heads, kv, dim, *lens, seed=64)
    check(run(ddm, x, causal, dim ** -0.5), *reference(x, causal, dim ** -0.5, dtype), ALL)
