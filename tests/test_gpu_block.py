"""Attention, rotary positions, norms and the gated layer together, as a block of the descriptor network runs them: in training
over packed images whose patches have rows and columns, and for single tokens over kept keys and values.

Each operator in 32 bits is within 64 roundings of 2^-24 of its value in the norm (their own tests); a block is ten of them in
a row and each may enlarge what came before it by its condition, here below four: 10 * 4 * 64 * 2^-24 = 1.5e-4.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

C, HEADS, KEY_HEADS, HIDDEN = 96, 6, 2, 168
D = C // HEADS


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


def weights(seed, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    p = dict(w0=1 + 0.1 * r(C), b0=0.1 * r(C), qkv=r((HEADS + 2 * KEY_HEADS) * D, C) / math.sqrt(C), out=r(C, C) / math.sqrt(C),
             scale1=0.3 + 0.1 * r(C), w1=1 + 0.1 * r(C), b1=0.1 * r(C), gated=r(2 * HIDDEN, C) / math.sqrt(C), bias=0.1 * r(2 * HIDDEN),
             down=r(C, HIDDEN) / math.sqrt(HIDDEN), bw=1 + 0.1 * r(C), bb=0.1 * r(C), w2=1 + 0.1 * r(C), b2=0.1 * r(C))
    return {n: t.to(dtype) for n, t in p.items()}


def block(ddm, x, gate, p, pos, freq, cu):
    h = ddm.layer_norm(x, p["w0"], p["b0"])
    qkv = (h @ p["qkv"].T).view(-1, HEADS + 2 * KEY_HEADS, D)
    q, k = ddm.rotary(qkv[:, :HEADS], qkv[:, HEADS:HEADS + KEY_HEADS], pos, freq)
    a = ddm.attention(q, k, qkv[:, HEADS + KEY_HEADS:], cu, cu)
    s, h = ddm.residual_norm(x, a.reshape(-1, C) @ p["out"].T, p["w1"], p["b1"], scale=p["scale1"])
    f = ddm.gated_linear(h, p["gated"], p["bias"]) @ p["down"].T
    return ddm.residual_norm(s, f, p["w2"], p["b2"], gate=gate, branch_norm=True, branch_weight=p["bw"], branch_bias=p["bb"])


def plain(x, gate, p, pos, freq, lens):
    norm = lambda z: (z - z.mean(1, keepdim=True)) * (z.var(1, unbiased=False, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    h = norm(x) * p["w0"] + p["b0"]
    qkv = (h @ p["qkv"].T).view(-1, HEADS + 2 * KEY_HEADS, D)
    axes, pairs = freq.shape
    angle = pos[:, :, None].double() * freq
    c, s = angle.cos()[:, None], angle.sin()[:, None]

    def turn(z):
        z = z.view(*z.shape[:2], axes, 2, pairs)
        a, b = z[..., 0, :], z[..., 1, :]
        return torch.stack((a * c - b * s, a * s + b * c), dim=-2).reshape(*z.shape[:2], D)

    q, k, v = turn(qkv[:, :HEADS]), turn(qkv[:, HEADS:HEADS + KEY_HEADS]), qkv[:, HEADS + KEY_HEADS:]
    outs, at = [], 0
    for n in lens:
        for_heads = []
        for head in range(HEADS):
            kh = head // (HEADS // KEY_HEADS)
            z = q[at:at + n, head] @ k[at:at + n, kh].T / math.sqrt(D)
            for_heads.append(torch.softmax(z, 1) @ v[at:at + n, kh])
        outs.append(torch.stack(for_heads, 1))
        at += n
    r = x + p["scale1"] * (torch.cat(outs).reshape(-1, C) @ p["out"].T)
    h = norm(r) * p["w1"] + p["b1"]
    g, u = (h @ p["gated"].T + p["bias"]).chunk(2, dim=1)
    f = (g * torch.sigmoid(g) * u) @ p["down"].T
    s2 = r + torch.sigmoid(gate) * (norm(f) * p["bw"] + p["bb"])
    return s2, norm(s2) * p["w2"] + p["b2"]


def test_a_block_in_training(ddm):
    shapes = [(5, 7), (9, 4), (1, 1)]
    lens = [h * w for h, w in shapes]
    pos = torch.cat([torch.cartesian_prod(torch.arange(h), torch.arange(w)) for h, w in shapes]).int().cuda()
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    freq = ddm.rotary_frequencies(D // 4, 100.0, device="cuda").expand(2, -1).contiguous()
    p = weights(1)
    torch.manual_seed(2)
    x, gate, ds, dy = (torch.randn(sum(lens), C, device="cuda") for _ in range(4))
    mine = {n: t.clone().requires_grad_() for n, t in dict(p, x=x, gate=gate).items()}
    s, y = block(ddm, mine["x"], mine["gate"], mine, pos, freq, cu)
    ((s * ds).sum() + (y * dy).sum()).backward()
    want = {n: t.double().requires_grad_() for n, t in dict(p, x=x, gate=gate).items()}
    ws, wy = plain(want["x"], want["gate"], want, pos, freq, lens)
    ((ws * ds.double()).sum() + (wy * dy.double()).sum()).backward()
    for name, a, b in [("s", s, ws), ("y", y, wy)] + [(n, mine[n].grad, want[n].grad) for n in mine]:
        off = ((a.double() - b).norm() / b.norm()).item()
        assert off <= 1.5e-4, (name, off)


def test_a_training_step_replayed_from_a_graph(ddm):
    """Forward and backward by the plain calls, captured once and replayed on other inputs; two graphs with workspaces of their own."""
    p = weights(3, torch.bfloat16)
    freq = ddm.rotary_frequencies(D // 2, device="cuda")
    pos = torch.arange(70, dtype=torch.int32, device="cuda")
    torch.manual_seed(4)
    x, dh = torch.randn(70, C, device="cuda").bfloat16(), torch.randn(70, HIDDEN, device="cuda").bfloat16()

    def step():
        y, mean, rstd = ddm.layer_norm_forward(x, p["w0"], p["b0"])
        q, _ = ddm.rotary_forward(y.view(70, HEADS, D), None, pos, freq)
        s, y, stats = ddm.residual_norm_forward(x, q.view(70, C), p["w1"], p["b1"], scale=p["scale1"])
        h, kept = ddm.gated_linear_forward(y, p["gated"], p["bias"], keep=True)
        dx, dw, db = ddm.gated_linear_backward(dh, y, p["gated"], kept)
        return (s, h, dx, dw, db) + ddm.residual_norm_backward(dx, None, x, q.view(70, C), stats, p["w1"], scale=p["scale1"])[:5]

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for i in range(3):
        x.copy_(torch.randn(70, C, device="cuda"))
        dh.copy_(torch.randn(70, HIDDEN, device="cuda"))
        want = step()
        for g, out in graphs:
            for t in out:
                t.fill_(7)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_single_tokens_over_kept_keys(ddm):
    """A token at a time over the keys and values kept so far gives what the whole sequence gives: every operator's rows are its
    own, and a causal query sees the same keys. In 32 bits; attention sums over keys in another order."""
    p, n = weights(5), 37
    freq = ddm.rotary_frequencies(D // 2, 10000.0, scaling="ramp", factor=4.0, length=64, device="cuda")
    torch.manual_seed(6)
    x = torch.randn(n, C, device="cuda")

    def rows(x, pos, keys=None):
        qkv = (ddm.layer_norm(x, p["w0"], p["b0"]) @ p["qkv"].T).view(-1, HEADS + 2 * KEY_HEADS, D)
        q, k = ddm.rotary_forward(qkv[:, :HEADS], qkv[:, HEADS:HEADS + KEY_HEADS], pos, freq, interleaved=True, magnitude=1.1)
        kv = torch.cat((k, qkv[:, HEADS + KEY_HEADS:]), 1)
        kv = kv if keys is None else torch.cat((keys, kv))
        a, _ = ddm.attention_forward(q, kv[:, :KEY_HEADS], kv[:, KEY_HEADS:], causal=True)
        s, h, _ = ddm.residual_norm_forward(x, a.reshape(-1, C) @ p["out"].T, p["w1"], p["b1"], scale=p["scale1"], rms=True)
        f, _ = ddm.gated_linear_forward(h, p["gated"], p["bias"], activation="gelu")
        return s + f @ p["down"].T, kv

    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    want, _ = rows(x, pos)
    keys = None
    for i in range(n):
        got, keys = rows(x[i:i + 1], pos[i:i + 1], keys)
        assert ((got - want[i:i + 1]).norm() / want[i].norm()).item() <= 1.5e-4, i
