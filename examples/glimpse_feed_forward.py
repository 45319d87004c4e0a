"""The feed-forward half of a transformer block over sampled glimpses, trained for a few steps.

A spatial transformer takes an affine glimpse of each feature map; its pixels become tokens x, and

    u = layer_norm(x),   z = (silu(u Wg^T) * (u Wu^T)) Wd^T,
    s = x + gate * layer_norm(z),   y = layer_norm(s),

with a gate per item, from a condition c of each: gate = c Wc.  Forward and backward passes call
the library's operators (the last three of the second line in one pass); Wd and Wc are plain
matrix products.  The parameters follow the gradient of the squared distance to a target:

    python examples/glimpse_feed_forward.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import spatial_transformer_sampling_gb300 as gs  # noqa: E402
from glimpse_block import glimpses  # noqa: E402


class FeedForward:
    """Parameters, and the state a forward pass keeps for the backward pass."""

    def __init__(self, channels, hidden, condition, dtype=torch.bfloat16, activation="silu", seed=0,
                 device="cuda"):
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        make = lambda *shape, std: (torch.randn(shape, generator=g) * std).to(device, dtype)
        one = lambda: torch.ones(channels, dtype=dtype, device=device)
        zero = lambda: torch.zeros(channels, dtype=dtype, device=device)
        std = channels ** -0.5
        self.activation = activation
        self.p = {"g0": one(), "b0": zero(), "Wg": make(hidden, channels, std=std),
                  "Wu": make(hidden, channels, std=std), "bg": make(hidden, std=0.1),
                  "bu": make(hidden, std=0.1), "Wd": make(channels, hidden, std=hidden ** -0.5),
                  "Wc": make(condition, channels, std=condition ** -0.5), "gz": one(), "bz": zero(),
                  "g1": one(), "b1": zero()}

    def forward(self, x, c):
        """x (N, L, C), c (N, condition) -> y (N, L, C)."""
        p, (N, L, C) = self.p, x.shape
        u, m0, i0 = gs.gs_layer_norm(x, p["g0"], p["b0"])
        h, G, U = gs.gs_gated_linear(u, p["Wg"], p["Wu"], p["bg"], p["bu"], self.activation, keep=True)
        z = (h.view(N * L, -1) @ p["Wd"].t()).view(N, L, C)
        gate = c @ p["Wc"]
        s, y, stats = gs.gs_residual_norm(x, z, p["g1"], p["b1"], gate=gate, z_scale=p["gz"],
                                          z_B=p["bz"])
        self.kept = (x, c, m0, i0, u, h, G, U, z, gate, s, stats)
        return y

    def backward(self, dy, ds=None):
        """Gradients of the parameters and of x for the last forward pass; ``ds`` is what reaches
        the residual stream otherwise."""
        x, c, m0, i0, u, h, G, U, z, gate, s, stats = self.kept
        p, grads, (N, L, C) = self.p, {}, x.shape
        back = gs.gs_residual_norm_backward(ds, dy, s, z, stats, p["g1"], bias=True, gate=gate,
                                            z_scale=p["gz"], z_B=p["bz"])
        grads.update(g1=back["dScale"], b1=back["dB"], gz=back["dz_scale"], bz=back["dz_B"])
        grads["Wc"] = c.t() @ back["dgate"]
        dz = back["dZ"].view(N * L, C)
        grads["Wd"] = dz.t() @ h.view(N * L, -1)
        dh = (dz @ p["Wd"]).view(h.shape)
        du, grads["Wg"], grads["Wu"], grads["bg"], grads["bu"] = gs.gs_gated_linear_backward(
            dh, u, p["Wg"], p["Wu"], G, U, self.activation, bias=True)
        dx, grads["g0"], grads["b0"] = gs.gs_layer_norm_backward(du, x, p["g0"], m0, i0)
        return grads, back["dX"] + dx


def train(steps=20, N=16, channels=64, hidden=172, condition=8, grid=(12, 16), dtype=torch.bfloat16,
          rate=0.1):
    g = torch.Generator(device="cpu")
    g.manual_seed(1)
    maps = torch.randn((N, channels, 32, 32), generator=g).to("cuda", dtype)
    theta = torch.eye(2, 3).repeat(N, 1, 1) + 0.1 * torch.randn((N, 2, 3), generator=g)
    tokens = glimpses(maps, theta.to("cuda", dtype), grid)
    c = torch.randn((N, condition), generator=g).to("cuda", dtype)
    target = tokens.float().mean(1, keepdim=True).expand_as(tokens)   # every token the mean one
    block, losses = FeedForward(channels, hidden, condition, dtype), []
    for _ in range(steps):
        off = block.forward(tokens, c).float() - target
        losses.append(off.square().mean().item())
        grads, _ = block.backward((off * (2.0 / channels / tokens.shape[1])).to(dtype))
        for name, d in grads.items():
            block.p[name] = (block.p[name].float() - rate * d.float()).to(dtype)
    return losses


if __name__ == "__main__":
    for step, loss in enumerate(train()):
        print(f"step {step:2d}  loss {loss:.4f}")
