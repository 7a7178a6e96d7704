"""Operators of a descriptor network and its training: packed attention, layer norm, matching loss.

The network that produces descriptor maps is a transformer over 16 x 16 pixel patches (a 512 x 384 image is 768
tokens) with a descriptor head trained by a symmetric softmax loss over matched descriptors. This file holds the
cases that time those operators, their plain forms in elementary torch operations, and their values in 64 bits.

Packed sets: sequences (or sets of matches) of different lengths lie one after another along the first axis, and
``cu`` (int32, number of sequences + 1) holds where each begins and the last ends.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def _lens(text):
    return [int(x) for x in text.split(",")]


def _text(lens):
    return ",".join(str(x) for x in lens)


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one pooled token of each image of a pair looks at its image's 768 patch tokens: the smallest call
        dict(name="attn-token-pair", op="attn", dtype="f16", heads=16, kv_heads=16, dim=64, lens_q="1,1",
             lens_k="768,768", causal=False, train=False),
        # one new token each over the keys of sequences of very different lengths, grouped heads
        dict(name="attn-token-long", op="attn", dtype="bf16", heads=32, kv_heads=8, dim=128, lens_q="1,1,1,1,1,1",
             lens_k="40001,16384,9000,2050,33,1", causal=True, train=False),
        # the encoder's self-attention over the 32 images of 16 pairs at 512 x 384
        dict(name="attn-encoder-16-pairs", op="attn", dtype="f16", heads=16, kv_heads=16, dim=64,
             lens_q=_text([768] * 32), lens_k=_text([768] * 32), causal=False, train=False),
        # whole prompts, causal, grouped heads, one of them empty and one of a single token
        dict(name="attn-prompts-causal", op="attn", dtype="bf16", heads=32, kv_heads=8, dim=128,
             lens_q="4096,3999,2500,1031,257,64,1,0", lens_k="4096,3999,2500,1031,257,64,1,0", causal=True, train=False),
        # the decoder's cross-attention in training: images of different shapes look at each other
        dict(name="attn-cross-train", op="attn", dtype="bf16", heads=12, kv_heads=12, dim=64,
             lens_q="768,1024,640,768,576,1000,768,901", lens_k="1024,768,768,640,1000,576,901,768", causal=False,
             train=True),
        # training on packed causal sequences with grouped heads
        dict(name="attn-causal-train", op="attn", dtype="bf16", heads=16, kv_heads=4, dim=128, lens_q="4096,3001,1024,513",
             lens_k="4096,3001,1024,513", causal=True, train=True),
        # layer norm over the tokens of one image pair, forward: a call among many small ones
        dict(name="norm-pair", op="norm", dtype="f16", wtype="f32", rows=1536, cols=1024, train=False),
        # layer norm in training over the tokens of 16 pairs
        dict(name="norm-train-16-pairs", op="norm", dtype="bf16", wtype="f32", rows=24576, cols=1024, train=True),
        # an odd width in 32 bits, rows that start off a 16-byte boundary
        dict(name="norm-train-odd", op="norm", dtype="f32", wtype="f32", rows=20011, cols=771, train=True),
        # the matching loss of one small image pair
        dict(name="match-small", op="match", dtype="f32", dim=24, lens="1000"),
        # the matching loss of 16 pairs with different numbers of matches
        dict(name="match-16-pairs", op="match", dtype="f16", dim=24,
             lens="4096,4001,3500,2900,2048,4096,4095,1777,333,4096,1,2500,3800,4096,3333,64"),
        # one pair with as many matches as a 512 x 512 map has stride-4 seeds
        dict(name="match-dense", op="match", dtype="bf16", dim=64, lens="16384"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    for _ in range(200):
        c = _draw(rng)
        if _cost(c) <= top and work(c)["flops"] > 0:
            return c
    return dict(listed()[0], dim=32)


def _draw(rng):
    op = rng.choice(["attn", "attn", "attn", "norm", "match"])
    if op == "norm":
        cols = _log_int(rng, 65, 4500)
        if rng.random() < 0.5:
            cols = -(-cols // 64) * 64
        dtype = rng.choice(["f32", "f16", "bf16"])
        return dict(op="norm", dtype=dtype, wtype=rng.choice(["f32", dtype]), cols=cols,
                    rows=_log_int(rng, 100, max(101, min(60000, 40_000_000 // cols))), train=rng.random() < 0.6)
    if op == "match":
        n = _log_int(rng, 200, 12000)
        lens = [n] + [_log_int(rng, 1, n) for _ in range(rng.randrange(0, 6))]
        rng.shuffle(lens)
        return dict(op="match", dtype=rng.choice(["f32", "f16", "bf16"]), dim=rng.choice([16, 24, 32, 48, 64, 128]),
                    lens=_text(lens))
    groups, kv = rng.choice([1, 1, 2, 4, 8]), rng.choice([1, 2, 4, 8, 12])
    dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    dim = rng.choice([32, 64, 64, 80, 128, 128])
    n, causal = rng.randrange(1, 9), rng.random() < 0.5
    if rng.random() < 0.35:                 # single tokens
        lens_k = [_log_int(rng, 30, 30000) for _ in range(n)]
        return dict(op="attn", dtype=dtype, heads=kv * groups, kv_heads=kv, dim=dim, lens_q=_text([1] * n),
                    lens_k=_text(lens_k), causal=causal, train=False)
    lens_k = [_log_int(rng, 17, 3500) for _ in range(n)]
    lens_q = lens_k if rng.random() < 0.6 else [_log_int(rng, 17, 3500) for _ in range(n)]
    return dict(op="attn", dtype=dtype, heads=kv * groups, kv_heads=kv, dim=dim, lens_q=_text(lens_q),
                lens_k=_text(lens_k), causal=causal, train=rng.random() < 0.5)


def _cost(c):
    """What a drawn case is held to: products of 32-bit inputs count eightfold, as their rate is far lower."""
    w = work(c)
    return w["flops"] * (8 if c["dtype"] == "f32" else 1) + 50 * w["bytes"]


def _visible(c):
    """Pairs of a query and a key that it may see, over all sequences."""
    total = 0
    for m, n in zip(_lens(c["lens_q"]), _lens(c["lens_k"])):
        if not c["causal"]:
            total += m * n
        else:                               # query i sees max(0, min(n, i + 1 + n - m)) keys
            first = max(0, m - n)
            total += sum((n - m + first + 1, n)) * (m - first) // 2 if m > first else 0
    return total


def work(c):
    e = _SIZE[c["dtype"]]
    if c["op"] == "attn":
        tq, tk = sum(_lens(c["lens_q"])), sum(_lens(c["lens_k"]))
        q, kv = tq * c["heads"] * c["dim"] * e, tk * c["kv_heads"] * c["dim"] * e
        flops = 4.0 * _visible(c) * c["heads"] * c["dim"]
        n = q + 2 * kv + q + 4 * tq * c["heads"]
        if c["train"]:                      # the gradient reads q, k, v, dout and writes dq, dk, dv
            n += q + q + 2 * kv
            flops *= 3.5
        return {"bytes": n, "flops": flops}
    if c["op"] == "norm":
        x, w = c["rows"] * c["cols"], c["cols"] * _SIZE[c["wtype"]]
        if c["train"]:                      # x and dy in, y and dx out
            return {"bytes": 4 * x * e + 8 * c["rows"] + 4 * w, "flops": 17.0 * x}
        return {"bytes": 2 * x * e + 8 * c["rows"] + 2 * w, "flops": 7.0 * x}
    lens = _lens(c["lens"])
    pairs, p = sum(n * n for n in lens), sum(lens)
    return {"bytes": 4 * p * c["dim"] * e + 16 * p, "flops": 6.0 * pairs * c["dim"]}


# ------------------------------------------------------------------------------------------------------- inputs
def _cu(lens, device):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=device)


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if c["op"] == "attn":
        lq, lk = _lens(c["lens_q"]), _lens(c["lens_k"])
        h, hk, d = c["heads"], c["kv_heads"], c["dim"]
        # keys share a mean, as a network's do; scores then spread by one to two around a common offset
        s = dict(c=c, q=(normal(sum(lq), h, d) * 1.3).to(dt), k=(normal(sum(lk), hk, d) + normal(1, hk, d)).to(dt),
                 v=normal(sum(lk), hk, d).to(dt), cu_q=_cu(lq, dev), cu_k=_cu(lk, dev), scale=d ** -0.5)
        if c["train"]:
            s["dout"] = normal(sum(lq), h, d).to(dt)
        return s
    if c["op"] == "norm":
        n, m = c["rows"], c["cols"]
        spread = normal(m).mul(0.7).exp()   # a residual stream: some channels are far larger than others
        s = dict(c=c, x=(normal(n, m) * spread + normal(m)).to(dt), weight=(1 + 0.2 * normal(m)).to(_DT[c["wtype"]]),
                 bias=(0.2 * normal(m)).to(_DT[c["wtype"]]), eps=1e-6)
        if c["train"]:
            s["dy"] = normal(n, m).to(dt)
        return s
    lens = _lens(c["lens"])
    p, d = sum(lens), c["dim"]
    a = torch.nn.functional.normalize(normal(p, d), dim=1)
    b = torch.nn.functional.normalize(a + 1.2 * normal(p, d) / math.sqrt(d), dim=1)
    # the loss is a mean over the matches, scaled up in float16 as training in that type does
    scale = (1024.0 if c["dtype"] == "f16" else 1.0) / p
    return dict(c=c, a=a.to(dt), b=b.to(dt), cu=_cu(lens, dev), temperature=0.07,
                dloss=(0.5 + torch.rand(p, generator=g, device=dev)) * scale)


# ------------------------------------------------------------------------------------------------- the two forms
def run(s):
    return {"attn": _attn, "norm": _norm, "match": _match}[s["c"]["op"]](s)


def _attn(s):
    c = s["c"]
    if own:
        import dense_descriptor_matching_amd as ddm
        out, lse = ddm.attention_forward(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"],
                                         scale=s["scale"])
        if not c["train"]:
            return {"out": out, "lse": lse}
        dq, dk, dv = ddm.attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu_q"], s["cu_k"],
                                            causal=c["causal"], scale=s["scale"])
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    lens_q, lens_k = _lens(c["lens_q"]), _lens(c["lens_k"])
    batch, m, n = len(lens_q), max(lens_q), max(lens_k)
    heads, kv, d = c["heads"], c["kv_heads"], c["dim"]
    groups, dt = heads // kv, s["q"].dtype
    at_q, in_q = _places(s["cu_q"], m)
    at_k, in_k = _places(s["cu_k"], n)

    def queries(x):         # packed [tokens, heads, d] to [batch * kv heads, group * m, d]
        x = x.float()[at_q].view(batch, m, kv, groups, d).permute(0, 2, 3, 1, 4)
        return x.reshape(batch * kv, groups * m, d)

    def keys(x):            # packed [tokens, kv heads, d] to [batch * kv heads, n, d]
        x = x.float()[at_k] * in_k[:, :, None, None]
        return x.permute(0, 2, 1, 3).reshape(batch * kv, n, d)

    def packed_q(x):
        return x.view(batch, kv, groups, m, d).permute(0, 3, 1, 2, 4).reshape(batch, m, heads, d)[in_q]

    def packed_k(x):
        return x.view(batch, kv, n, d).permute(0, 2, 1, 3)[in_k]

    q, k, v = queries(s["q"]), keys(s["k"]), keys(s["v"])
    see = in_q[:, :, None] & in_k[:, None, :]
    if c["causal"]:
        i, j = torch.arange(m, device=q.device), torch.arange(n, device=q.device)
        last = i[None, :] + (s["cu_k"].diff() - s["cu_q"].diff()).long()[:, None]
        see = see & (j[None, None, :] <= last[:, :, None])
    see = see[:, None, None]
    p = torch.bmm(q, k.transpose(1, 2)).mul_(s["scale"]).view(batch, kv, groups, m, n)
    p.masked_fill_(~see, float("-inf"))
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).permute(0, 3, 1, 2, 4).reshape(batch, m, heads)[in_q]
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    p = p.view(batch * kv, groups * m, n)
    out = torch.bmm(p, v)
    got = {"out": packed_q(out).to(dt), "lse": lse}
    if not c["train"]:
        return got
    dout = queries(s["dout"])
    dout = dout.view(batch, kv, groups, m, d).mul(in_q[:, None, None, :, None]).view(batch * kv, groups * m, d)
    got["dv"] = packed_k(torch.bmm(p.transpose(1, 2), dout)).to(dt)
    delta = (dout * out).sum(-1, keepdim=True)
    p.mul_(torch.bmm(dout, v.transpose(1, 2)).sub_(delta)).mul_(s["scale"])
    got["dq"] = packed_q(torch.bmm(p, k)).to(dt)
    got["dk"] = packed_k(torch.bmm(p.transpose(1, 2), q)).to(dt)
    return got


def _places(cu, most):
    """Where the tokens of each sequence, padded to `most`, lie in the packed tensor, and which of them are its own."""
    cu = cu.long()
    i = torch.arange(most, device=cu.device)
    at = cu[:-1, None] + i
    return torch.minimum(at, cu[-1] - 1), i < cu.diff()[:, None]


def _norm(s):
    c = s["c"]
    if own:
        import dense_descriptor_matching_amd as ddm
        y, mean, rstd = ddm.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=s["eps"])
        if not c["train"]:
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = ddm.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)
        return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dweight": dw, "dbias": db}
    dt = s["x"].dtype
    x, w = s["x"].float(), s["weight"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = (x.square().mean(1, keepdim=True) + s["eps"]).rsqrt()
    x = x * rstd
    got = {"y": (x * w + s["bias"].float()).to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if not c["train"]:
        return got
    dy = s["dy"].float()
    got["dweight"] = (dy * x).sum(0).to(s["weight"].dtype)
    got["dbias"] = dy.sum(0).to(s["weight"].dtype)
    dy = dy * w
    got["dx"] = ((dy - dy.mean(1, keepdim=True) - x * (dy * x).mean(1, keepdim=True)) * rstd).to(dt)
    return got


def _match(s):
    if own:
        import dense_descriptor_matching_amd as ddm
        loss, lse_a, lse_b = ddm.matching_loss_forward(s["a"], s["b"], s["cu"], temperature=s["temperature"])
        da, db = ddm.matching_loss_backward(s["dloss"], s["a"], s["b"], lse_a, lse_b, s["cu"],
                                            temperature=s["temperature"])
        return {"loss": loss, "lse_a": lse_a, "lse_b": lse_b, "da": da, "db": db}
    dt, t = s["a"].dtype, s["temperature"]
    lens = _lens(s["c"]["lens"])
    at, mine = _places(s["cu"], max(lens))
    a, b = (x.float()[at] * mine[:, :, None] for x in (s["a"], s["b"]))
    g = s["dloss"][at] * mine
    score = torch.bmm(a, b.transpose(1, 2)) / t
    score.masked_fill_(~(mine[:, :, None] & mine[:, None, :]), float("-inf"))
    top_a, top_b = (score.amax(k, keepdim=True) for k in (2, 1))
    top_a, top_b = (torch.where(x == float("-inf"), torch.zeros_like(x), x) for x in (top_a, top_b))
    lse_a = (score - top_a).exp().sum(2, keepdim=True).log() + top_a
    lse_b = (score - top_b).exp().sum(1, keepdim=True).log() + top_b
    hit = torch.diagonal(score, dim1=1, dim2=2)
    loss = 0.5 * (lse_a[:, :, 0] - hit + lse_b[:, 0] - hit)
    # the gradient by the score: half of g_i softmax over row i and g_j softmax over column j, less g on the diagonal
    d = (score - lse_a).exp_().mul_(0.5 * g[:, :, None])
    d = torch.where(mine[:, :, None], d, torch.zeros_like(d))
    e = (score - lse_b).exp_().mul_(0.5 * g[:, None, :])
    d += torch.where(mine[:, None, :], e, torch.zeros_like(e))
    torch.diagonal(d, dim1=1, dim2=2).sub_(g)
    d /= t
    da, db = torch.bmm(d, b), torch.bmm(d.transpose(1, 2), a)
    return {"loss": loss[mine], "lse_a": lse_a[:, :, 0][mine], "lse_b": lse_b[:, 0][mine], "da": da[mine].to(dt),
            "db": db[mine].to(dt)}


# ---------------------------------------------------------------------------------------------- values in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    f8 = torch.float64
    if c["op"] == "norm":
        x = s["x"].to(f8)
        mu = x.sum(1) / c["cols"]
        var = ((x - mu[:, None]) ** 2).sum(1) / c["cols"]
        r = 1.0 / torch.sqrt(var + s["eps"])
        xhat = (x - mu[:, None]) * r[:, None]
        w = s["weight"].to(f8)
        got = {"y": xhat * w + s["bias"].to(f8), "mean": mu, "rstd": r}
        if c["train"]:
            dy = s["dy"].to(f8)
            got["dweight"], got["dbias"] = torch.einsum("nc,nc->c", dy, xhat), dy.sum(0)
            u = dy * w
            got["dx"] = r[:, None] * (u - (u.sum(1) / c["cols"])[:, None]
                                      - xhat * (torch.einsum("nc,nc->n", u, xhat) / c["cols"])[:, None])
        return got
    if c["op"] == "match":
        got = {k: [] for k in ("loss", "lse_a", "lse_b", "da", "db")}
        at = 0
        for n in _lens(c["lens"]):
            if n == 0:
                continue
            a, b, g = (s[k][at:at + n].to(f8) for k in ("a", "b", "dloss"))
            at += n
            z = a @ b.T / s["temperature"]
            la, lb = torch.logsumexp(z, 1), torch.logsumexp(z, 0)
            got["loss"].append((la + lb) / 2 - z.diagonal())
            got["lse_a"].append(la)
            got["lse_b"].append(lb)
            dz = (torch.exp(z - la[:, None]) * g[:, None] + torch.exp(z - lb[None, :]) * g[None, :]) / 2
            dz = (dz - torch.diag(g)) / s["temperature"]
            got["da"].append(dz @ b)
            got["db"].append(dz.T @ a)
        return {k: torch.cat(v) for k, v in got.items()}
    heads, groups = c["heads"], c["heads"] // c["kv_heads"]
    q, k, v = (s[x].to(f8) for x in ("q", "k", "v"))
    got = {"out": torch.zeros_like(q), "lse": q.new_full(q.shape[:2], -math.inf)}
    if c["train"]:
        dout = s["dout"].to(f8)
        got.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    i0 = j0 = 0
    for m, n in zip(_lens(c["lens_q"]), _lens(c["lens_k"])):
        rows, cols = slice(i0, i0 + m), slice(j0, j0 + n)
        i0, j0 = i0 + m, j0 + n
        if m == 0 or n == 0:
            continue
        hidden = None
        if c["causal"]:
            hidden = torch.ones(m, n, dtype=torch.bool, device=q.device).triu(n - m + 1)
        for h in range(heads):
            z = q[rows, h] @ k[cols, h // groups].T * s["scale"]
            if hidden is not None:
                z[hidden] = -math.inf
            lse = torch.logsumexp(z, 1)
            p = torch.exp(z - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
            got["lse"][rows, h] = lse
            got["out"][rows, h] = p @ v[cols, h // groups]
            if c["train"]:
                do = dout[rows, h]
                got["dv"][cols, h // groups] += p.T @ do
                dp = do @ v[cols, h // groups].T
                dz = p * (dp - (p * dp).sum(1)[:, None]) * s["scale"]
                got["dq"][rows, h] = dz @ k[cols, h // groups]
                got["dk"][cols, h // groups] += dz.T @ q[rows, h]
    return got
