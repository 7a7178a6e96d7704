"""Attention over packed sequences against its definition in 64 bits.

Tolerances are bounds per element, computed from the same 64-bit quantities. With u the unit roundoff of the inputs' type
(2^-8 bfloat16, 2^-11 float16, 0 float32, whose roundings the fp32 term covers) the kernels round each probability P and each
dS = P (dP - D) once to that type before its product, each output once, and take D from the rounded out:
  out: u (sum P|v| + |out|)        dv: u (sum P|do| + |dv|)
  dq:  u (scale sum |dS||k| + |dq|) + scale sum P dD |k|,  dD_i = 2 u sum_d |do|(|o| + sum P|v|);  dk likewise
fp16 also holds nothing below 2^-24: half of that for each rounded P (times |v|) and, relative to the row's largest |do|,
for each dS. fp32 accumulation and the exponentials add (n + 8 max|z| + 16) 2^-24 of the same absolute sums. A factor 1.25
covers products of the terms.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


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


def make(dtype, heads, kv, dim, lens_q, lens_k, seed=0, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    tq, tk = sum(lens_q) + 2 * pad, sum(lens_k) + 2 * pad
    return dict(q=(r(tq, heads, dim) * 1.3).to(DT[dtype]), k=(r(tk, kv, dim) + r(1, kv, dim)).to(DT[dtype]),
                v=r(tk, kv, dim).to(DT[dtype]), dout=r(tq, heads, dim).to(DT[dtype]), cu_q=cu_of(lens_q, pad),
                cu_k=cu_of(lens_k, pad))


def reference(x, causal, scale, dtype):
    """Values and bounds in 64 bits, sequence by sequence and head by head."""
    q, k, v, do = (x[n].double() for n in ("q", "k", "v", "dout"))
    u, tiny = U[dtype], TINY[dtype]
    names = ("out", "dq", "dk", "dv")
    val = dict(out=torch.zeros_like(q), lse=torch.full(q.shape[:2], -math.inf, device="cuda", dtype=torch.float64),
               dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(k))
    tol = {n: torch.zeros_like(val[n]) for n in names}
    tol["lse"] = torch.zeros_like(val["lse"])
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
        for h in range(q.shape[1]):
            c = h // group
            z = (q[i, h] @ k[j, c].T) * scale
            zm = z.masked_fill(~see, -math.inf)
            lse = torch.logsumexp(zm, 1)
            p = torch.exp(zm - lse.masked_fill(lse == -math.inf, 0)[:, None])
            any_ = see.any(1)
            big = float(z[see].abs().max()) if bool(see.any()) else 0.0
            e = (max(m * group, n) + 8 * big + 16) * 2.0 ** -24
            va, ka, qa, da = v[j, c].abs(), k[j, c].abs(), q[i, h].abs(), do[i, h].abs()
            o = p @ v[j, c]
            pv = p @ va
            dp = do[i, h] @ v[j, c].T
            d = (do[i, h] * o).sum(1)
            ds = p * (dp - d[:, None])
            # what rounding and the 32-bit sums do to P, D and dS
            vis = see.double()
            d_err = 2 * (u + e) * (da * (o.abs() + pv)).sum(1) + (2 * tiny * (da * (vis @ va)).sum(1) if tiny else 0)
            row = da.amax(1)
            ds_err = (u + 2 * e) * ds.abs() + p * (d_err + 2 * e * (da @ va.T + d.abs()[:, None]).amax(1))[:, None] \
                + 4 * tiny * row[:, None] * vis
            p_err = (u + 2 * e) * p + tiny * vis
            val["lse"][i, h], val["out"][i, h] = lse, o
            tol["lse"][i, h] = torch.where(any_, e * (1 + lse.abs()), torch.zeros_like(lse))
            tol["out"][i, h] = p_err @ va + u * o.abs()
            val["dq"][i, h] = scale * ds @ k[j, c]
            tol["dq"][i, h] = scale * ds_err @ ka
            val["dk"][j, c] += scale * ds.T @ q[i, h]
            tol["dk"][j, c] += scale * ds_err.T @ qa
            val["dv"][j, c] += p.T @ do[i, h]
            tol["dv"][j, c] += p_err.T @ da
    for n in ("dq", "dk", "dv"):
        tol[n] += u * val[n].abs()
    if tiny:                                # outputs below fp16's normal range
        for n in names:
            tol[n] += tiny
    return val, tol


def check(got, val, tol, names):
    for n in names:
        a, b, t = got[n].double(), val[n], 1.25 * tol[n]
        inf = b == -math.inf
        assert torch.equal(a == -math.inf, inf), n
        off = (a - b).abs().masked_fill(inf, 0) - t
        assert not torch.isnan(a).any(), n
        assert off.max().item() <= 0, (n, off.max().item(), t.max().item()) if off.numel() else n


def run(ddm, x, causal, scale, backward=True):
    out, lse = ddm.attention_forward(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], causal=causal, scale=scale)
    got = dict(out=out, lse=lse)
    if backward:
        got["dq"], got["dk"], got["dv"] = ddm.attention_backward(
            x["dout"], x["q"], x["k"], x["v"], out, lse, x["cu_q"], x["cu_k"], causal=causal, scale=scale)
    return got


ALL = ("out", "lse", "dq", "dk", "dv")
LENS = [((1,), (1,)), ((5, 70), (5, 70)), ((64, 128, 129), (64, 128, 129)), ((200, 33, 0, 1), (130, 300, 5, 0)),
        ((31, 257), (33, 300)), ((300,), (40,)), ((700, 3), (700, 900))]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("heads,kv,dim", [(2, 2, 64), (8, 2, 128)])
def test_values_and_gradients(ddm, dtype, causal, lens, heads, kv, dim):
    x = make(dtype, heads, kv, dim, *lens, seed=len(lens[0]) + dim)
    check(run(ddm, x, causal, dim ** -0.5), *reference(x, causal, dim ** -0.5, dtype), ALL)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("heads,kv,dim", [(3, 1, 16), (5, 5, 24), (2, 1, 32), (6, 6, 40), (12, 4, 80), (7, 1, 96),
                                          (16, 8, 8), (24, 8, 120)])
def test_head_layouts(ddm, dtype, heads, kv, dim):
    x = make(dtype, heads, kv, dim, (65, 17), (65, 97), seed=3)
    check(run(ddm, x, True, 0.2), *reference(x, True, 0.2, dtype), ALL)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [((1, 1), (768, 768)), ((1,), (5000,)), ((1, 1, 1, 1), (3000, 64, 1, 0)),
                                  ((1, 0, 2), (1000, 300, 129)), ((1, 0, 2, 1, 1), (9000, 2000, 1290, 0, 1)), ((3, 40, 1), (2000, 100, 900)), ((2, 90, 1, 1), (700, 800, 3000, 5))])
@pytest.mark.parametrize("heads,kv,dim", [(4, 4, 64), (16, 2, 128), (6, 2, 24)])
def test_few_rows_over_long_keys(ddm, dtype, causal, lens, heads, kv, dim):
    x = make(dtype, heads, kv, dim, *lens, seed=11)
    check(run(ddm, x, causal, dim ** -0.5), *reference(x, causal, dim ** -0.5, dtype), ALL)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [((40, 90), (70, 33)), ((1, 1), (900, 700))])
def test_tokens_outside_every_sequence(ddm, dtype, lens):
    """Infinities and NaN before and after the sequences reach nothing, and those tokens' own outputs are zeros."""
    pad = 9
    x = make(dtype, 4, 2, 64, *lens, seed=5, pad=pad)
    val, tol = reference(x, True, 0.125, dtype)
    for n in ("q", "k", "v", "dout"):
        x[n][:pad], x[n][-pad:] = float("nan"), float("inf")
    got = run(ddm, x, True, 0.125)
    check(got, val, tol, ALL)
    for n in ("out", "dq", "dk", "dv"):
        assert (got[n][:pad] == 0).all() and (got[n][-pad:] == 0).all()


def test_neighbouring_sequence_reaches_nothing(ddm):
    """A sequence of NaN leaves its neighbours as they are, although tiles of 64 keys and rows hold several sequences."""
    x = make("bf16", 4, 2, 64, (40, 30, 50), (40, 30, 50), seed=6)
    a = run(ddm, x, False, 0.125)
    for n in ("q", "k", "v", "dout"):
        x[n][40:70] = float("nan")
    b = run(ddm, x, False, 0.125)
    for n in ("out", "dq", "dk", "dv"):
        assert torch.equal(a[n][:40], b[n][:40]) and torch.equal(a[n][70:], b[n][70:])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_strided_views(ddm, dtype):
    """q, k, v as views of one packed projection, and heads before tokens, give what contiguous copies give."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    qkv = torch.randn(333, 8 + 2 + 2, 64, generator=g, device="cuda").to(DT[dtype])
    cu = cu_of((100, 233))
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    dout = torch.randn(8, 333, 64, generator=g, device="cuda").to(DT[dtype]).transpose(0, 1)
    a = run(ddm, dict(q=q, k=k, v=v, dout=dout, cu_q=cu, cu_k=cu), True, 0.125)
    c = [t.contiguous() for t in (q, k, v, dout)]
    b = run(ddm, dict(q=c[0], k=c[1], v=c[2], dout=c[3], cu_q=cu, cu_k=cu), True, 0.125)
    for n in ALL:
        assert torch.equal(a[n], b[n])


@pytest.mark.parametrize("lens_q", [(1,), (200,)])
def test_keys_beyond_32_bit_offsets(ddm, lens_q):
    """Keys spread over 6 GB: token stride 2 MB."""
    n, step = 3000, 1 << 20
    buf = torch.zeros(n * step, dtype=torch.bfloat16, device="cuda")
    x = make("bf16", 4, 1, 128, lens_q, (n,), seed=2)
    k = buf.view(n, step)[:, :128].unflatten(1, (1, 128))
    v = buf.view(n, step)[:, 128:256].unflatten(1, (1, 128))
    k.copy_(x["k"])
    v.copy_(x["v"])
    a = run(ddm, x, True, 0.09)
    b = run(ddm, dict(x, k=k, v=v), True, 0.09)
    for m in ALL:
        assert torch.equal(a[m], b[m])


def test_large_scores(ddm):
    """Scores in the thousands: the largest wins without overflow."""
    x = make("f32", 2, 2, 64, (70,), (130,), seed=4)
    x["q"] *= 40
    val, tol = reference(x, False, 1.0, "f32")
    check(run(ddm, x, False, 1.0), val, tol, ("out", "lse"))


def test_small_gradients_in_half_precision(ddm):
    """Gradients far below fp16's normal range inside the products: dS is scaled by its row before it is rounded."""
    x = make("f16", 4, 2, 64, (300, 20), (300, 20), seed=8)
    x["dout"] *= 2.0 ** -10
    check(run(ddm, x, False, 0.125), *reference(x, False, 0.125, "f16"), ALL)


def test_single_sequence_without_boundaries(ddm):
    x = make("bf16", 4, 2, 64, (150,), (150,), seed=9)
    a = run(ddm, x, True, 0.125)
    b = run(ddm, dict(x, cu_q=None, cu_k=None), True, 0.125)
    for n in ALL:
        assert torch.equal(a[n], b[n])


def test_many_short_sequences(ddm):
    lens = [(i * 7) % 23 for i in range(150)]
    x = make("bf16", 4, 4, 64, lens, lens, seed=10)
    check(run(ddm, x, True, 0.125), *reference(x, True, 0.125, "bf16"), ALL)


def test_bad_boundaries_stay_inside(ddm):
    """Boundaries outside the tensor or out of order are clamped: any result, no access outside (the values are checked by
    the clamped equivalent where there is one)."""
    x = make("bf16", 2, 2, 64, (50, 50), (50, 50), seed=12)
    bad = torch.tensor([-5, 50, 1000], dtype=torch.int32, device="cuda")
    a = run(ddm, dict(x, cu_q=bad, cu_k=bad), False, 0.125)
    b = run(ddm, x, False, 0.125)
    for n in ALL:
        assert torch.equal(a[n], b[n])


@pytest.mark.parametrize("cu", [[0, 90, 30, 100], [100, 0, 100, 0], [50, 40, 30, 20], [0, 100, 100, 0]])
@pytest.mark.parametrize("lens", [((30, 30, 40), (30, 30, 40)), ((1, 0, 1), (400, 300, 500))])
def test_boundaries_out_of_order_stay_inside(ddm, cu, lens):
    """Decreasing boundaries give no defined values, but no length below zero and no place before a tensor: the calls end, and
    later ones are right."""
    x = make("bf16", 2, 2, 64, *lens, seed=18)
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    run(ddm, dict(x, cu_q=bad, cu_k=bad), True, 0.125)
    torch.cuda.synchronize()
    good = run(ddm, x, True, 0.125)
    check(good, *reference(x, True, 0.125, "bf16"), ALL)


def test_heads_far_apart(ddm):
    """Heads before tokens, 18 MB from one head to the next."""
    g = torch.Generator(device="cuda")
    g.manual_seed(19)
    k, v = (torch.randn(2, 70000, 128, generator=g, device="cuda").bfloat16().transpose(0, 1) for _ in range(2))
    x = make("bf16", 4, 2, 128, (100,), (100,), seed=19)
    far = dict(x, k=k, v=v, cu_q=None, cu_k=None)
    near = dict(far, k=k.contiguous(), v=v.contiguous())
    a, b = run(ddm, far, False, 0.09), run(ddm, near, False, 0.09)
    for n in ALL:
        assert torch.equal(a[n], b[n])


def test_same_bits_every_time_and_on_a_side_stream(ddm):
    x = make("bf16", 8, 2, 128, (500, 300), (500, 300), seed=13)
    a = run(ddm, x, True, 0.09)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run(ddm, x, True, 0.09)
    s.synchronize()
    for n in ALL:
        assert torch.equal(a[n], b[n])


@pytest.mark.parametrize("lens", [((500, 300), (500, 300)), ((1, 1), (3000, 300))])
def test_graph_replays(ddm, lens):
    x = make("f16", 8, 2, 64, *lens, seed=14)
    want = run(ddm, x, True, 0.125)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(ddm, x, True, 0.125)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ddm, x, True, 0.125)
    for _ in range(3):
        for t in got.values():
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for n in ALL:
            assert torch.equal(got[n], want[n])


def test_gradient_against_differences(ddm):
    """Central differences of a fixed functional of out, in float32: rounding 2^-24 sum|w out| / step against the third
    derivative times step^2 leaves some 1e-3 of the gradient's norm at step 1e-2."""
    x = make("f32", 4, 2, 32, (20, 9), (20, 15), seed=15)
    got = run(ddm, x, True, 0.2)
    f = lambda y: (run(ddm, y, True, 0.2, False)["out"].double() * x["dout"].double()).sum().item()  # noqa: E731
    g = torch.Generator(device="cuda")
    g.manual_seed(16)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        w = torch.randn(x[n].shape, generator=g, device="cuda")
        h = 1e-2 / w.norm().item() * math.sqrt(w.numel())
        diff = (f(dict(x, **{n: x[n] + h * w})) - f(dict(x, **{n: x[n] - h * w}))) / (2 * h)
        want = (got[d].double() * w.double()).sum().item()
        assert abs(diff - want) <= 2e-3 * got[d].double().norm().item() * w.double().norm().item() / math.sqrt(w.numel()) + 1e-3


def test_autograd(ddm):
    x = make("bf16", 4, 2, 64, (70, 33), (70, 33), seed=17)
    want = run(ddm, x, True, 64 ** -0.5)
    q, k, v = (x[n].clone().requires_grad_() for n in ("q", "k", "v"))
    out = ddm.attention(q, k, v, x["cu_q"], x["cu_k"], causal=True)
    out.backward(x["dout"])
    assert torch.equal(out, want["out"])
    for t, n in ((q, "dq"), (k, "dk"), (v, "dv")):
        assert torch.equal(t.grad, want[n])
    ddm.attention(q, k, v, x["cu_q"], x["cu_k"], causal=True).sum().backward()     # an expanded gradient


def test_refusals(ddm):
    x = make("bf16", 4, 2, 64, (8,), (8,))
    q, k, v, cu = x["q"], x["k"], x["v"], x["cu_q"]
    f = ddm.attention_forward
    with pytest.raises(TypeError):
        f(q.cpu(), k, v)
    with pytest.raises(TypeError):
        f(q, k.float(), v)
    with pytest.raises(TypeError):
        f(q.double(), k.double(), v.double())
    with pytest.raises(ValueError):
        f(q[:, :3], k, v)                              # 3 query heads over 2 key heads
    with pytest.raises(ValueError):
        f(q, k, v[:7])
    with pytest.raises(ValueError):
        f(q, k, v, cu)                                 # one of the two boundaries
    with pytest.raises(ValueError):
        f(q, k, v, cu, torch.cat([cu, cu[-1:]]))
    with pytest.raises(TypeError):
        f(q, k, v, cu.long(), cu)
    with pytest.raises(ValueError):
        f(q.transpose(1, 2).contiguous().transpose(1, 2), k, v)      # head dimension not contiguous
    with pytest.raises(ValueError):
        f(torch.zeros(8 * 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(8, 4, 64), k, v)   # 8-byte boundary
    with pytest.raises(ddm.DDMError):
        f(q, k, v, scale=0.0)
    with pytest.raises(ddm.DDMError):
        f(q, k, v, scale=float("nan"))
    for dim in (12, 136):
        t = torch.zeros(4, 1, dim, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(ddm.DDMError) as e:
            f(t, t, t)
        assert e.value.status == -4
    out, lse = f(q, k, v)
    with pytest.raises(ValueError):
        ddm.attention_backward(x["dout"][:7], q, k, v, out, lse)
    with pytest.raises(TypeError):
        ddm.attention_backward(x["dout"], q, k, v, out, lse.double())


def test_nothing_to_do(ddm):
    z = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    x = make("bf16", 4, 2, 64, (8,), (8,))
    out, lse = ddm.attention_forward(z, x["k"], x["v"])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = ddm.attention_forward(x["q"], x["k"][:0], x["v"][:0])
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = ddm.attention_backward(x["dout"], x["q"], x["k"][:0], x["v"][:0], out, lse)
    assert (dq == 0).all() and dk.shape == dv.shape == (0, 2, 64)
    dq, dk, dv = ddm.attention_backward(z, z, x["k"], x["v"], z, torch.zeros(0, 4, device="cuda"))
    assert dq.shape == (0, 4, 64) and (dk == 0).all() and (dv == 0).all()
