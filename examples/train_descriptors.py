"""Trains a small descriptor network on synthetic image pairs and matches with what it learned.

    python examples/train_descriptors.py [--steps 60]

Two images of different sizes show the same random texture at a shift, each under its own noise and beside as many channels that
say nothing, three times as loud: untrained descriptors are mostly those. A transformer over all their
pixels (packed: the images' tokens lie one after another) gives every pixel a unit-norm descriptor: self-attention within each
image, cross-attention to the other one, layer norms between, as in MASt3R's encoder and decoder in small. The matching loss
over known matches trains it; Fast Reciprocal Matching then matches the two descriptor maps. Everything but the plain matrix
products and the optimizer runs in this package's kernels.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_descriptor_matching_amd as ddm  # noqa: E402

CHANNELS, HEADS, KEY_HEADS, D_DESC = 128, 4, 2, 24


class Block(torch.nn.Module):
    """Layer norm, attention with grouped heads and a residual; then layer norm, MLP and a residual."""

    def __init__(self, cross: bool):
        super().__init__()
        self.cross = cross
        dim = CHANNELS // HEADS
        self.q = torch.nn.Linear(CHANNELS, HEADS * dim)
        self.kv = torch.nn.Linear(CHANNELS, 2 * KEY_HEADS * dim)
        self.out = torch.nn.Linear(CHANNELS, CHANNELS)
        self.mlp = torch.nn.Sequential(torch.nn.Linear(CHANNELS, 2 * CHANNELS), torch.nn.GELU(),
                                       torch.nn.Linear(2 * CHANNELS, CHANNELS))
        self.weight = torch.nn.Parameter(torch.ones(2, CHANNELS))
        self.bias = torch.nn.Parameter(torch.zeros(2, CHANNELS))

    def forward(self, x, cu, sizes):
        h = ddm.layer_norm(x, self.weight[0], self.bias[0])
        other, cu_k = h, cu
        if self.cross:                      # sequence 0 looks at image 2's tokens and sequence 1 at image 1's
            a, b = h.split(sizes)
            other, cu_k = torch.cat([b, a]), (cu[-1] - cu).flip(0).contiguous()
        dim = CHANNELS // HEADS
        q = self.q(h).bfloat16().view(-1, HEADS, dim)
        kv = self.kv(other).bfloat16().view(-1, 2 * KEY_HEADS, dim)      # keys and values are views of one projection
        y = ddm.attention(q, kv[:, :KEY_HEADS], kv[:, KEY_HEADS:], cu, cu_k)
        x = x + self.out(y.reshape(-1, CHANNELS).float())
        return x + self.mlp(ddm.layer_norm(x, self.weight[1], self.bias[1]))


class DescriptorNet(torch.nn.Module):
    def __init__(self, features: int):
        super().__init__()
        self.embed = torch.nn.Linear(features, CHANNELS)
        self.blocks = torch.nn.ModuleList([Block(False), Block(True)])
        self.weight = torch.nn.Parameter(torch.ones(CHANNELS))
        self.bias = torch.nn.Parameter(torch.zeros(CHANNELS))
        self.head = torch.nn.Linear(CHANNELS, D_DESC)

    def forward(self, tokens, cu, sizes):
        x = self.embed(tokens)
        for block in self.blocks:
            x = block(x, cu, sizes)
        return torch.nn.functional.normalize(self.head(ddm.layer_norm(x, self.weight, self.bias)), dim=1)


def make_pair(shape1, shape2, shift, features, noise, generator, device):
    """Tokens of both images, and the linear pixels (i, j) that show the same place: (x, y) in image 1 is (x + dx, y + dy)
    of the texture, whose corner is image 2's."""
    (h1, w1), (h2, w2), (dx, dy) = shape1, shape2, shift
    H, W = max(h1 + dy, h2), max(w1 + dx, w2)
    texture = torch.randn(H, W, features, generator=generator, device=device)
    def seen(part):
        h, w, _ = part.shape
        own = torch.randn(h, w, 2 * features, generator=generator, device=device)
        return torch.cat([part + noise * own[..., :features], 3 * own[..., features:]], dim=2)

    a, b = seen(texture[dy:dy + h1, dx:dx + w1]), seen(texture[:h2, :w2])
    y, x = torch.meshgrid(torch.arange(h1, device=device), torch.arange(w1, device=device), indexing="ij")
    both = (y + dy < h2) & (x + dx < w2)
    return a.reshape(h1 * w1, -1), b.reshape(h2 * w2, -1), (y * w1 + x)[both], ((y + dy) * w2 + x + dx)[both]


def train(steps: int = 60, seed: int = 0, device="cuda", shape1=(24, 18), shape2=(20, 22), features=16, noise=0.2, log=print):
    """Returns (first loss, last loss, share of true matches among those found on an unseen pair, how many were found)."""
    torch.manual_seed(seed)
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    net = DescriptorNet(2 * features).to(device)
    optimizer = torch.optim.AdamW(net.parameters(), lr=2e-3)
    n1, n2 = shape1[0] * shape1[1], shape2[0] * shape2[1]
    cu = torch.tensor([0, n1, n1 + n2], dtype=torch.int32, device=device)
    first = last = None
    for step in range(steps):
        a, b, i, j = make_pair(shape1, shape2, (3, 2), features, noise, g, device)
        d1, d2 = net(torch.cat([a, b]), cu, (n1, n2)).split((n1, n2))
        loss = ddm.matching_loss(d1[i], d2[j], temperature=0.07).mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        last = loss.item()
        first = last if first is None else first
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step}: matching loss {last:.4f}")
    with torch.no_grad():
        a, b, i, j = make_pair(shape1, shape2, (3, 2), features, noise, g, device)
        d1, d2 = net(torch.cat([a, b]), cu, (n1, n2)).half().split((n1, n2))
        fi, fj, _ = ddm.frm_match(d1.reshape(*shape1, -1).contiguous(), d2.reshape(*shape2, -1).contiguous(), 2, 10)
    truth = torch.full((n1,), -1, dtype=torch.int64, device=device)
    truth[i] = j
    share = (truth[fi.long()] == fj.long()).float().mean().item() if len(fi) else 0.0
    log(f"{len(fi)} reciprocal matches on an unseen pair, {100 * share:.1f}% of them true")
    return first, last, share, len(fi)


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    parser.add_argument("--steps", type=int, default=60)
    parser.add_argument("--seed", type=int, default=0)
    args = parser.parse_args()
    train(args.steps, args.seed)
