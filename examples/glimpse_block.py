"""A transformer block over sampled glimpses, trained for a few steps.

A spatial transformer takes an affine glimpse of each feature map (gs_affine_sample); its h x w
pixels become tokens of one block

    a = x + dropout(attention(layer_norm(x)) Wo),   y = layer_norm(a)

whose attention has a learned bias by relative grid position.  Forward and backward passes call
the library's operators; the projections are plain matrix products.  The parameters follow the
gradient of the squared distance to a target, and the loss goes down:

    python examples/glimpse_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spatial_transformer_sampling_gb300 as gs  # noqa: E402


class GlimpseBlock:
    """Parameters, and the state a forward pass keeps for the backward pass."""

    def __init__(self, channels, heads, grid, dtype=torch.bfloat16, ratio=0.1, seed=0, device="cuda"):
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        make = lambda *shape, std: (torch.randn(shape, generator=g) * std).to(device, dtype)
        self.grid, self.heads, self.ratio, self.seed = grid, heads, ratio, seed
        self.buckets, rows = gs.gs_relative_buckets(grid, grid, num_buckets=8, max_distance=16,
                                                    device=device)
        ones = torch.ones(channels, dtype=dtype, device=device)
        self.p = {"g1": ones, "b1": torch.zeros_like(ones), "g2": ones.clone(),
                  "b2": torch.zeros_like(ones), "Wqkv": make(channels, 3 * channels, std=0.05),
                  "Wo": make(channels, channels, std=0.05), "table": make(rows, heads, std=0.02)}

    def forward(self, x, step):
        """x (N, L, C) -> y (N, L, C)."""
        N, L, C = x.shape
        p, H = self.p, self.heads
        u, m1, i1 = gs.gs_layer_norm(x, p["g1"], p["b1"])
        qkv = (u.view(N * L, C) @ p["Wqkv"]).view(N, L, 3, H, C // H)
        q, k, v = qkv.unbind(2)
        o, lse = gs.gs_attention(q, k, v, p["table"], self.buckets, self.grid, self.grid)
        branch = (o.view(N * L, C) @ p["Wo"]).view(N, L, C)
        a = gs.gs_dropout(branch, self.ratio, self.seed, step, residual=x)
        y, m2, i2 = gs.gs_layer_norm(a, p["g2"], p["b2"])
        self.kept = (x, m1, i1, u, qkv, o, lse, a, m2, i2, step)
        return y

    def backward(self, dy):
        """Gradients of the parameters and of x for the last forward pass."""
        x, m1, i1, u, qkv, o, lse, a, m2, i2, step = self.kept
        N, L, C = x.shape
        p, grads = self.p, {}
        da, grads["g2"], grads["b2"] = gs.gs_layer_norm_backward(dy, a, p["g2"], m2, i2)
        dbranch = gs.gs_dropout(da, self.ratio, self.seed, step).view(N * L, C)   # the same mask
        grads["Wo"] = o.view(N * L, C).t() @ dbranch
        do = (dbranch @ p["Wo"].t()).view(o.shape)
        q, k, v = qkv.unbind(2)
        dq, dk, dv, grads["table"] = gs.gs_attention_backward(
            do, q, k, v, o, lse, p["table"], self.buckets, self.grid, self.grid)
        dqkv = torch.stack((dq, dk, dv), 2).view(N * L, 3 * C)
        grads["Wqkv"] = u.view(N * L, C).t() @ dqkv
        du = (dqkv @ p["Wqkv"].t()).view(N, L, C)
        dx, grads["g1"], grads["b1"] = gs.gs_layer_norm_backward(du, x, p["g1"], m1, i1)
        return grads, da + dx


def glimpses(maps, theta, grid):
    """Affine glimpses of feature maps (N, C, H, W) as tokens (N, h * w, C)."""
    size = (maps.shape[0], maps.shape[1]) + tuple(grid)
    sampled = gs.gs_affine_sample(theta, size, maps, "linear", "border", 1)
    return sampled.flatten(2).transpose(1, 2).contiguous()


def train(steps=20, N=16, channels=64, heads=4, grid=(12, 16), dtype=torch.bfloat16, rate=0.1):
    g = torch.Generator(device="cpu")
    g.manual_seed(1)
    maps = torch.randn((N, channels, 32, 32), generator=g).to("cuda", dtype)
    theta = torch.eye(2, 3).repeat(N, 1, 1) + 0.1 * torch.randn((N, 2, 3), generator=g)
    tokens = glimpses(maps, theta.to("cuda", dtype), grid)
    target = tokens.float().mean(1, keepdim=True).expand_as(tokens)   # every token the mean one
    block, losses = GlimpseBlock(channels, heads, grid, dtype), []
    for step in range(steps):
        off = block.forward(tokens, step).float() - target
        losses.append(off.square().mean().item())
        grads, _ = block.backward((off * (2.0 / channels / tokens.shape[1])).to(dtype))
        for name, d in grads.items():
            block.p[name] = (block.p[name].float() - rate * d.float()).to(dtype)
    return losses


if __name__ == "__main__":
    for step, loss in enumerate(train()):
        print(f"step {step:2d}  loss {loss:.4f}")
