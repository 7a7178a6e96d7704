"""Operators of a descriptor network's blocks: rotary positions, residual norm, gated linear layer.

A block of the transformer that produces descriptor maps rotates its queries and keys by the places of their tokens,
adds what attention gives to the residual stream between two norms, and passes the result through a gated linear
layer. This file holds the cases that time those operators, their plain forms in elementary torch operations, and
their values in 64 bits. A 512 x 384 image is 32 x 24 = 768 tokens of 16 x 16 pixels.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token each of six long sequences, interleaved pairs, frequencies scaled for long contexts
        dict(name="rotary-tokens", op="rotary", dtype="bf16", tokens=6, heads=32, kv_heads=8, dim=128, axes=1, pairs=64,
             interleaved=True, far=60000, factor=8.0, train=False),
        # the encoder's queries and keys of 16 pairs at 512 x 384, placed by patch row and column, in training
        dict(name="rotary-train-16-pairs", op="rotary", dtype="bf16", tokens=24576, heads=16, kv_heads=16, dim=64, axes=2,
             pairs=16, interleaved=False, far=32, factor=1.0, train=True),
        # whole long prompts, grouped heads, half of each head rotated, interleaved
        dict(name="rotary-prompts-part", op="rotary", dtype="f16", tokens=40001, heads=32, kv_heads=8, dim=128, axes=1,
             pairs=32, interleaved=True, far=0, factor=1.0, train=False),
        # two pooled tokens between attention and the next product: the smallest call
        dict(name="norm-tokens", op="norm", dtype="f16", wtype="f16", rows=2, cols=1024, rms=False, scale=True, gate=False,
             branch_norm=False, train=False),
        # the tokens of one image pair, with the branch's learned scale, forward
        dict(name="norm-pair", op="norm", dtype="f16", wtype="f32", rows=1536, cols=1024, rms=False, scale=True, gate=False,
             branch_norm=False, train=False),
        # training over the tokens of 16 pairs with everything: norm of the branch, its gate and its scale
        dict(name="norm-train-16-pairs", op="norm", dtype="bf16", wtype="f32", rows=24576, cols=1024, rms=False, scale=True,
             gate=True, branch_norm=True, train=True),
        # an odd width in 32 bits without means, norms before and after, no gate
        dict(name="norm-train-odd-rms", op="norm", dtype="f32", wtype="f32", rows=10007, cols=1285, rms=True, scale=False,
             gate=False, branch_norm=True, train=True),
        # one pooled token of each image of a pair: the weights' bytes count
        dict(name="gated-tokens", op="gated", dtype="bf16", rows=2, cols=1024, hidden=2736, act="silu", bias=True, train=False),
        # single tokens of a batch of sequences, a hidden width that no tile divides
        dict(name="gated-batch-odd", op="gated", dtype="f16", rows=37, cols=2048, hidden=5461, act="silu", bias=False, train=False),
        # the encoder's feed-forward over the tokens of one image pair
        dict(name="gated-pair", op="gated", dtype="f16", rows=1536, cols=1024, hidden=2736, act="gelu", bias=True, train=False),
        # the same in training over the tokens of 16 pairs
        dict(name="gated-train-16-pairs", op="gated", dtype="bf16", rows=24576, cols=1024, hidden=2736, act="silu", bias=True,
             train=True),
        # a small odd one in training in 32 bits
        dict(name="gated-train-odd", op="gated", dtype="f32", rows=2001, cols=771, hidden=1030, act="gelu", bias=True, train=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    for _ in range(200):
        c = _draw(rng)
        if _cost(c) <= top:
            return c
    return dict(listed()[0], tokens=7)


def _draw(rng):
    op = rng.choice(["rotary", "norm", "gated", "gated"])
    dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    if op == "rotary":
        kv = rng.choice([1, 2, 4, 8, 12])
        heads = kv * rng.choice([1, 1, 2, 4])
        dim = rng.choice([20, 32, 64, 64, 80, 96, 128, 128])
        axes = rng.choice([1, 1, 2, 2, 3])
        most = dim // (2 * axes)
        pairs = rng.choice([most, most, max(1, most // 2), rng.randrange(1, most + 1)])
        return dict(op="rotary", dtype=dtype, tokens=_log_int(rng, 1, 50000), heads=heads, kv_heads=kv, dim=dim, axes=axes,
                    pairs=pairs, interleaved=rng.random() < 0.5, far=_log_int(rng, 1, 1000000),
                    factor=rng.choice([1.0, 1.0, 4.0]), train=rng.random() < 0.5)
    if op == "norm":
        cols = _log_int(rng, 65, 4500)
        if rng.random() < 0.5:
            cols = -(-cols // 64) * 64
        return dict(op="norm", dtype=dtype, wtype=rng.choice(["f32", dtype]), cols=cols,
                    rows=_log_int(rng, 1, max(2, min(40000, 30_000_000 // cols))), rms=rng.random() < 0.4,
                    scale=rng.random() < 0.6, gate=rng.random() < 0.4, branch_norm=rng.random() < 0.5, train=rng.random() < 0.6)
    cols, hidden = _log_int(rng, 64, 4100), _log_int(rng, 64, 8200)
    if rng.random() < 0.6:
        cols, hidden = -(-cols // 64) * 64, -(-hidden // 16) * 16
    return dict(op="gated", dtype=dtype, rows=_log_int(rng, 1, 20000), cols=cols, hidden=hidden,
                act=rng.choice(["silu", "silu", "gelu", "sigmoid"]), bias=rng.random() < 0.6, train=rng.random() < 0.5)


def _cost(c):
    """What a drawn case is held to: products of 32-bit inputs count eightfold, as their rate is far lower."""
    w = work(c)
    return w["flops"] * (8 if c["dtype"] == "f32" else 1) + 50 * w["bytes"]


def work(c):
    e = _SIZE[c["dtype"]]
    if c["op"] == "rotary":
        x = c["tokens"] * (c["heads"] + c["kv_heads"]) * c["dim"]
        pairs = c["tokens"] * (c["heads"] + c["kv_heads"]) * c["axes"] * c["pairs"]
        both = 2 if c["train"] else 1       # the gradient rotates dq and dk back
        return {"bytes": both * 2 * x * e + 4 * c["tokens"] * c["axes"] + 8 * c["axes"] * c["pairs"], "flops": both * 6.0 * pairs}
    if c["op"] == "norm":
        x, n = c["rows"] * c["cols"], 4 if c["branch_norm"] else 2
        params = (2 + 2 * c["branch_norm"] + c["scale"]) * c["cols"] * _SIZE[c["wtype"]]
        moved, flops = 4 + c["gate"], (10 + 8 * c["branch_norm"] + 6 * c["gate"]) * x
        if c["train"]:                      # dy and ds in, dx, dbranch and dgate out, with the parameters' gradients
            moved, flops, params = moved + 4 + c["gate"], 2.5 * flops, 2 * params
        return {"bytes": moved * x * e + 4 * n * c["rows"] + params, "flops": float(flops)}
    n, cols, f = c["rows"], c["cols"], c["hidden"]
    x, w, h = n * cols, 2 * f * cols, n * f
    b = 2 * f if c["bias"] else 0
    if c["train"]:                          # dh in, dx and the gradients of weight and bias out
        return {"bytes": 2 * (x + w + h + b) * e, "flops": 6.0 * n * w}
    return {"bytes": (x + w + h + b) * e, "flops": 2.0 * n * w}


# ------------------------------------------------------------------------------------------------------- inputs
def _frequencies(c):
    """f_i = base^(-i / pairs), for long contexts divided by the factor where a pair turns less than once in the length
    trained on, unchanged where it turns 32 times or more, and between them in proportion."""
    f = (100.0 if c["axes"] > 1 else 10000.0) ** (-torch.arange(c["pairs"], dtype=torch.float64) / c["pairs"])
    if c["factor"] != 1.0:
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f * keep + f / c["factor"] * (1 - keep)
    return f


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if c["op"] == "rotary":
        t, h, hk, d = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        if c["axes"] == 1 and c["far"] == 0:    # a whole prompt
            places = torch.arange(t, device=dev)
        else:                                   # patches of images, or where each sequence has got to
            places = torch.randint(0, max(c["far"], 1), (t, c["axes"]), generator=g, device=dev)
            places = places[:, 0].contiguous() if c["axes"] == 1 else places
        s = dict(c=c, q=normal(t, h, d).to(dt), k=(normal(t, hk, d) + normal(1, hk, d)).to(dt), positions=places.int(),
                 frequencies=_frequencies(c).expand(c["axes"], -1).contiguous().to(dev),
                 magnitude=0.1 * math.log(c["factor"]) + 1.0)
        if c["train"]:
            s["dq"], s["dk"] = normal(t, h, d).to(dt), normal(t, hk, d).to(dt)
        return s
    if c["op"] == "norm":
        n, m, wt = c["rows"], c["cols"], _DT[c["wtype"]]
        spread = normal(m).mul(0.7).exp()   # a residual stream: some channels are far larger than others
        s = dict(c=c, x=(normal(n, m) * spread + normal(m)).to(dt), branch=(0.8 * normal(n, m) + 0.3 * normal(m)).to(dt),
                 weight=(1 + 0.2 * normal(m)).to(wt), bias=(0.2 * normal(m)).to(wt), eps=1e-6, scale=None, gate=None,
                 branch_weight=None, branch_bias=None)
        if c["scale"]:
            s["scale"] = (0.3 + 0.1 * normal(m)).to(wt)
        if c["gate"]:
            s["gate"] = (1.5 * normal(n, m)).to(dt)
        if c["branch_norm"]:
            s["branch_weight"], s["branch_bias"] = (1 + 0.2 * normal(m)).to(wt), (0.2 * normal(m)).to(wt)
        if c["train"]:
            s["dy"], s["ds"] = normal(n, m).to(dt), normal(n, m).to(dt)
        return s
    n, m, f = c["rows"], c["cols"], c["hidden"]
    # what a norm gives, and weights whose projections then spread by about one
    s = dict(c=c, x=normal(n, m).to(dt), weight=(normal(2 * f, m) / math.sqrt(m)).to(dt), bias=None)
    if c["bias"]:
        s["bias"] = (0.2 * normal(2 * f)).to(dt)
    if c["train"]:
        s["dh"] = normal(n, f).to(dt)
    return s


# ------------------------------------------------------------------------------------------------- the two forms
def run(s):
    return {"rotary": _rotary, "norm": _norm, "gated": _gated}[s["c"]["op"]](s)


def _rotary(s):
    c = s["c"]
    if own:
        import dense_descriptor_matching_amd as ddm
        how = dict(interleaved=c["interleaved"], magnitude=s["magnitude"])
        q, k = ddm.rotary_forward(s["q"], s["k"], s["positions"], s["frequencies"], **how)
        if not c["train"]:
            return {"q": q, "k": k}
        dq, dk = ddm.rotary_backward(s["dq"], s["dk"], s["positions"], s["frequencies"], **how)
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    angle = s["positions"].view(-1, c["axes"], 1).double() * s["frequencies"]           # [tokens, axes, pairs]
    cos, sin = (s["magnitude"] * f(angle).float()[:, None] for f in (torch.cos, torch.sin))
    used = 2 * c["axes"] * c["pairs"]

    def turn(x, sin):
        y = x.float().clone()
        shape = (c["pairs"], 2) if c["interleaved"] else (2, c["pairs"])
        p = y[..., :used].reshape(*y.shape[:2], c["axes"], *shape)
        a, b = p.unbind(-1 if c["interleaved"] else -2)
        p = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1 if c["interleaved"] else -2)
        y[..., :used] = p.reshape(*y.shape[:2], used)
        return y.to(x.dtype)

    got = {"q": turn(s["q"], sin), "k": turn(s["k"], sin)}
    if c["train"]:
        got["dq"], got["dk"] = turn(s["dq"], -sin), turn(s["dk"], -sin)
    return got


def _norm(s):
    c = s["c"]
    if own:
        import dense_descriptor_matching_amd as ddm
        how = dict(scale=s["scale"], gate=s["gate"], branch_norm=c["branch_norm"], branch_weight=s["branch_weight"],
                   branch_bias=s["branch_bias"], rms=c["rms"])
        r, y, stats = ddm.residual_norm_forward(s["x"], s["branch"], s["weight"], s["bias"], eps=s["eps"], **how)
        got = {"s": r, "y": y, "stats": stats}
        if c["train"]:
            grads = ddm.residual_norm_backward(s["dy"], s["ds"], s["x"], s["branch"], stats, s["weight"], **how)
            names = ("dx", "dbranch", "dweight", "dbias", "dscale", "dgate", "dbranch_weight", "dbranch_bias")
            got.update((n, g) for n, g in zip(names, grads) if g is not None)
        return got
    dt, wt = s["x"].dtype, s["weight"].dtype

    def normed(x):
        mean = torch.zeros_like(x[:, :1]) if c["rms"] else x.mean(1, keepdim=True)
        x = x - mean
        rstd = (x.square().mean(1, keepdim=True) + s["eps"]).rsqrt()
        return x * rstd, mean[:, 0], rstd

    def unnormed(u, x, rstd):                # the gradient through x = normed(...)
        u = u if c["rms"] else u - u.mean(1, keepdim=True)
        return (u - x * (u * x).mean(1, keepdim=True)) * rstd

    t = s["branch"].float()
    if c["branch_norm"]:
        branch, branch_mean, branch_rstd = normed(t)
        t = branch * s["branch_weight"].float() + s["branch_bias"].float()
    open_ = 1.0 / (1.0 + (-s["gate"].float()).exp()) if c["gate"] else None
    part = t * open_ if c["gate"] else t
    r = s["x"].float() + (part * s["scale"].float() if c["scale"] else part)
    x, mean, rstd = normed(r)
    got = {"s": r.to(dt), "y": (x * s["weight"].float() + s["bias"].float()).to(dt)}
    stats = [mean, rstd[:, 0]] + ([branch_mean, branch_rstd[:, 0]] if c["branch_norm"] else [])
    got["stats"] = torch.stack(stats)
    if not c["train"]:
        return got
    dy = s["dy"].float()
    got["dweight"], got["dbias"] = (dy * x).sum(0).to(wt), dy.sum(0).to(wt)
    dr = s["ds"].float() + unnormed(dy * s["weight"].float(), x, rstd)
    got["dx"] = dr.to(dt)
    if c["scale"]:
        got["dscale"] = (dr * part).sum(0).to(wt)
        dr = dr * s["scale"].float()
    if c["gate"]:
        got["dgate"] = (dr * t * open_ * (1 - open_)).to(dt)
        dr = dr * open_
    if c["branch_norm"]:
        got["dbranch_weight"], got["dbranch_bias"] = (dr * branch).sum(0).to(wt), dr.sum(0).to(wt)
        dr = unnormed(dr * s["branch_weight"].float(), branch, branch_rstd)
    got["dbranch"] = dr.to(dt)
    return got


def _gated(s):
    c = s["c"]
    if own:
        import dense_descriptor_matching_amd as ddm
        h, kept = ddm.gated_linear_forward(s["x"], s["weight"], s["bias"], activation=c["act"], keep=c["train"])
        if not c["train"]:
            return {"h": h}
        dx, dw, db = ddm.gated_linear_backward(s["dh"], s["x"], s["weight"], kept, activation=c["act"], need_dbias=c["bias"])
        return {"h": h, "dx": dx, "dweight": dw, "dbias": db} if c["bias"] else {"h": h, "dx": dx, "dweight": dw}
    dt, f = s["x"].dtype, c["hidden"]
    x, w = s["x"].float(), s["weight"].float()
    p = x @ w.T
    if c["bias"]:
        p = p + s["bias"].float()
    g, u = p[:, :f], p[:, f:]
    act, slope = _activation(g, c["act"])
    got = {"h": (act * u).to(dt)}
    if not c["train"]:
        return got
    dh = s["dh"].float()
    dp = torch.cat((dh * u * slope, dh * act), dim=1)
    got["dx"], got["dweight"] = (dp @ w).to(dt), (dp.T @ x).to(dt)
    if c["bias"]:
        got["dbias"] = dp.sum(0).to(dt)
    return got


def _activation(g, kind):
    """The activation of g and its derivative."""
    if kind == "gelu":
        below = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * below, below + g * (-0.5 * g * g).exp() * (1 / math.sqrt(2 * math.pi))
    t = 1.0 / (1.0 + (-g).exp())
    return (t, t * (1 - t)) if kind == "sigmoid" else (g * t, t * (1 + g * (1 - t)))


# ---------------------------------------------------------------------------------------------- values in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return {"rotary": _exact_rotary, "norm": _exact_norm, "gated": _exact_gated}[c["op"]](c, s)


def _exact_rotary(c, s):
    at = s["positions"].view(c["tokens"], c["axes"])

    def turned(x, sign):
        y = x.clone()
        for axis in range(c["axes"]):
            angle = at[:, axis, None].double() * s["frequencies"][axis]
            z = torch.polar(torch.full_like(angle, s["magnitude"]), sign * angle)[:, None]
            first = 2 * c["pairs"] * axis
            even = slice(first, first + 2 * c["pairs"], 2) if c["interleaved"] else slice(first, first + c["pairs"])
            odd = (slice(first + 1, first + 2 * c["pairs"], 2) if c["interleaved"]
                   else slice(first + c["pairs"], first + 2 * c["pairs"]))
            z = z * torch.complex(x[..., even].contiguous(), x[..., odd].contiguous())
            y[..., even], y[..., odd] = z.real, z.imag
        return y

    got = {"q": turned(s["q"], 1), "k": turned(s["k"], 1)}
    if c["train"]:
        got["dq"], got["dk"] = turned(s["dq"], -1), turned(s["dk"], -1)
    return got


def _exact_norm(c, s):
    def stats(x):
        mu = x.new_zeros(len(x)) if c["rms"] else x.sum(1) / c["cols"]
        return mu, 1.0 / torch.sqrt(((x - mu[:, None]) ** 2).sum(1) / c["cols"] + s["eps"])

    def back(u, x, mu, rstd):
        xhat = (x - mu[:, None]) * rstd[:, None]
        out = u - xhat * (torch.einsum("nc,nc->n", u, xhat) / c["cols"])[:, None]
        if not c["rms"]:
            out = out - (u.sum(1) / c["cols"])[:, None]
        return out * rstd[:, None]

    t, all_stats = s["branch"], []
    if c["branch_norm"]:
        bm, br = stats(s["branch"])
        bhat = (s["branch"] - bm[:, None]) * br[:, None]
        t, all_stats = bhat * s["branch_weight"] + s["branch_bias"], [bm, br]
    factor = torch.ones_like(t) if s["scale"] is None else s["scale"].expand_as(t)
    sig = torch.sigmoid(s["gate"]) if c["gate"] else torch.ones_like(t)
    r = s["x"] + factor * sig * t
    m, rstd = stats(r)
    rhat = (r - m[:, None]) * rstd[:, None]
    got = {"s": r, "y": rhat * s["weight"] + s["bias"], "stats": torch.stack([m, rstd] + all_stats)}
    if c["train"]:
        got["dweight"], got["dbias"] = torch.einsum("nc,nc->c", s["dy"], rhat), s["dy"].sum(0)
        dr = s["ds"] + back(s["dy"] * s["weight"], r, m, rstd)
        got["dx"] = dr
        if c["scale"]:
            got["dscale"] = torch.einsum("nc,nc->c", dr, sig * t)
        if c["gate"]:
            got["dgate"] = dr * factor * t * torch.sigmoid(s["gate"]) * torch.sigmoid(-s["gate"])
        dt = dr * factor * sig
        if c["branch_norm"]:
            got["dbranch_weight"], got["dbranch_bias"] = torch.einsum("nc,nc->c", dt, bhat), dt.sum(0)
            dt = back(dt * s["branch_weight"], s["branch"], bm, br)
        got["dbranch"] = dt
    return got


def _exact_gated(c, s):
    wg, wu = s["weight"].chunk(2)
    bg, bu = s["bias"].chunk(2) if c["bias"] else (0.0, 0.0)
    g, u = s["x"] @ wg.T + bg, s["x"] @ wu.T + bu
    if c["act"] == "gelu":
        phi = torch.special.ndtr(g)
        a, d = g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:
        t = torch.sigmoid(g)
        a, d = (t, t * torch.sigmoid(-g)) if c["act"] == "sigmoid" else (g * t, t + g * t * torch.sigmoid(-g))
    got = {"h": a * u}
    if c["train"]:
        dg, du = s["dh"] * u * d, s["dh"] * a
        got["dx"] = dg @ wg + du @ wu
        got["dweight"] = torch.cat((dg.T @ s["x"], du.T @ s["x"]))
        if c["bias"]:
            got["dbias"] = torch.cat((dg.sum(0), du.sum(0)))
    return got
