"""Attention in 16 bits: the norm of each output's error against 64 bits.

A bound for each element adds all roundings with their worst signs and is far above what they come to. Here they are taken
as independent and uniform within half a unit in the last place: of a value x that is at most u |x| / sqrt 3 (root of the
mean square; u = 2^-8 bfloat16, 2^-11 float16), below float16's normal range 2^-25 / sqrt 3. Squares add up. Rounded are
P (before its products with v and do), dS = P (do.v - D) (before those with k and q; in float16 in units of at most twice the
largest |do|) and the outputs; D_i = do_i.o_i carries the roundings of o_i into all dS of its row at once:
  out: sum P^2 v^2 + out^2            dv: sum P^2 do^2 + dv^2
  dq:  scale^2 (sum dS^2 |k|^2 + sum_i var D_i |sum_j P_ij k_j|^2) + dq^2,   dk: scale^2 (sum dS^2 + P^2 var D_i) |q|^2 + dk^2
times u^2 / 3, with var D_i = sum_d do^2 (o^2 + sum_j P^2 v^2). With 10^4 and more elements the norm strays from its
expectation by a few per cent; a factor of 1.25 covers that and the 32-bit sums.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import DT, TINY, U, ddm, make, run  # noqa: E402,F401  (ddm is a fixture)

ALL = ("out", "dq", "dk", "dv")


def reference(x, causal, scale, dtype):
    """64-bit values, and the expected square of each output's error norm."""
    q, k, v, do = (x[n].double() for n in ("q", "k", "v", "dout"))
    r2, t2 = U[dtype] ** 2 / 3, TINY[dtype] ** 2 / 3
    val = dict(out=torch.zeros_like(q), dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    sq = dict.fromkeys(ALL, 0.0)
    cq, ck = x["cu_q"].tolist(), x["cu_k"].tolist()
    group = q.shape[1] // k.shape[1]
    for b in range(len(cq) - 1):
        i, j = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        m, n = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        if m == 0 or n == 0:
            continue
        see = torch.ones(m, n, dtype=torch.bool, device="cuda")
        if causal:
            see = see.tril(n - m)
        vis = see.double()
        for h in range(q.shape[1]):
            c = h // group
            qh, kh, vh, dh = q[i, h], k[j, c], v[j, c], do[i, h]
            z = (qh @ kh.T * scale).masked_fill(~see, -math.inf)
            lse = torch.logsumexp(z, 1)
            p = torch.exp(z - lse.masked_fill(lse == -math.inf, 0)[:, None])
            o = p @ vh
            ds = p * (dh @ vh.T - (dh * o).sum(1)[:, None])
            p_var = r2 * p ** 2 + t2 * vis
            o_var = p_var @ vh ** 2 + r2 * o ** 2
            d_var = (dh ** 2 * o_var).sum(1)
            ds_var = r2 * ds ** 2 + 4 * t2 * dh.abs().max() ** 2 * vis
            val["out"][i, h], val["dq"][i, h] = o, scale * ds @ kh
            val["dk"][j, c] += scale * ds.T @ qh
            val["dv"][j, c] += p.T @ dh
            sq["out"] += float((p_var @ vh ** 2).sum())
            sq["dv"] += float((p_var.T @ dh ** 2).sum())
            sq["dq"] += scale ** 2 * float((ds_var @ kh ** 2).sum() + (d_var[:, None] * (p @ kh) ** 2).sum())
            sq["dk"] += scale ** 2 * float(((ds_var + p ** 2 * d_var[:, None]).T @ qh ** 2).sum())
    for n in ALL:
        sq[n] += float((r2 * val[n] ** 2 + t2).sum())
    return val, sq


def check(got, val, sq):
    for n in ALL:
        off = float((got[n].double() - val[n]).norm())
        assert off <= 1.25 * math.sqrt(sq[n]), (n, off / float(val[n].norm()), math.sqrt(sq[n]) / float(val[n].norm()))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads,kv,dim", [(2, 2, 64), (4, 4, 32)])
@pytest.mark.parametrize("offset", [2, 20, 100])
def test_first_keys_unlike_the_rest(ddm, dtype, causal, heads, kv, dim, offset):
    """A few keys (tokens at a sequence's start, say) lie far from the others where no query looks: they weigh little in P,
    and nothing of them may reach the gradients of rows that attend elsewhere."""
    x = make(dtype, heads, kv, dim, (1024, 300), (1024, 300), seed=21)
    x["q"][:, :, 0] = -x["q"][:, :, 0].abs() - 1
    for first in (0, 1024):
        x["k"][first:first + 8, :, 0] += offset
    check(run(ddm, x, causal, dim ** -0.5), *reference(x, causal, dim ** -0.5, dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mean", [0.0, 1.0, 5.0])
def test_half_of_the_keys_far_away(ddm, dtype, mean):
    """Keys in two clusters, of which the queries attend one."""
    x = make(dtype, 4, 2, 64, (700,), (900,), seed=22)
    x["q"][:, :, 0] = -x["q"][:, :, 0].abs() - 1
    x["k"][::2, :, 0] += 40
    x["k"][:, :, 1:] += mean
    check(run(ddm, x, False, 0.125), *reference(x, False, 0.125, dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [((700, 3), (700, 900)), ((300, 257), (333, 300)), ((900,), (130,))])
@pytest.mark.parametrize("heads,kv,dim", [(2, 2, 64), (8, 2, 128), (6, 3, 80), (12, 1, 32), (4, 4, 24)])
def test_errors_add_up_as_roundings_do(ddm, dtype, causal, lens, heads, kv, dim):
    x = make(dtype, heads, kv, dim, *lens, seed=23)
    check(run(ddm, x, causal, dim ** -0.5), *reference(x, causal, dim ** -0.5, dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** 6])
def test_gradients_of_other_sizes(ddm, dtype, size):
    """What float16 cannot hold of dS is that far below its row's largest, not below 2^-24."""
    x = make(dtype, 4, 2, 64, (500, 300), (500, 300), seed=24)
    x["dout"] = x["dout"] * size
    check(run(ddm, x, True, 0.125), *reference(x, True, 0.125, dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv", [(40, 1), (71, 1), (128, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_groups_larger_than_a_tile(ddm, dtype, heads, kv, dim):
    x = make(dtype, heads, kv, dim, (70, 33), (70, 40), seed=25)
    check(run(ddm, x, True, dim ** -0.5), *reference(x, True, dim ** -0.5, dtype))
