"""The example's transformer block on the GPU: its gradients against 64-bit automatic
differentiation of the same formulas, and its training loss."""
import importlib.util
import os

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "glimpse_block.py")


@pytest.fixture(scope="module")
def example(gs_cuda):
    spec = importlib.util.spec_from_file_location("glimpse_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _formula(p, x, dy, mask, buckets, grid, H, eps=1e-5):
    """Gradients of sum(y * dy) in 64 bits by automatic differentiation."""
    leaf = {k: v.detach().double().cpu().requires_grad_(True) for k, v in p.items()}
    x = x.detach().double().cpu().requires_grad_(True)
    N, L, C = x.shape

    def norm(t, g, b):
        c = t - t.mean(2, keepdim=True)
        return c / torch.sqrt((c * c).mean(2, keepdim=True) + eps) * g + b

    u = norm(x, leaf["g1"], leaf["b1"])
    q, k, v = (u @ leaf["Wqkv"]).view(N, L, 3, H, C // H).permute(2, 0, 3, 1, 4)
    _, which = ref.pair_bias(p["table"].cpu(), buckets, grid, grid)
    s = q @ k.transpose(2, 3) * (C // H) ** -0.5 + leaf["table"][which].permute(2, 0, 1)
    o = (torch.softmax(s, 3) @ v).permute(0, 2, 1, 3).reshape(N, L, C)
    a = x + (o @ leaf["Wo"]) * mask
    y = norm(a, leaf["g2"], leaf["b2"])
    (y * dy.double().cpu()).sum().backward()
    return y.detach(), {k: t.grad for k, t in leaf.items()}, x.grad


def test_block_gradients_match_automatic_differentiation(example, gs_cuda):
    N, C, H, grid = 3, 32, 2, (6, 7)
    block = example.GlimpseBlock(C, H, grid, torch.float32, ratio=0.25, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for name in ("g1", "b1", "g2", "b2"):
        block.p[name] = block.p[name] + 0.1 * torch.randn(C, generator=g, device="cuda")
    maps = torch.randn((N, C, 20, 20), generator=g, device="cuda")
    theta = torch.eye(2, 3, device="cuda").repeat(N, 1, 1) * 0.7
    x = example.glimpses(maps, theta, grid)
    dy = torch.randn(x.shape, generator=g, device="cuda")
    y = block.forward(x, 11)
    grads, dx = block.backward(dy)
    mask = gs_cuda.gs_dropout(torch.ones_like(x), 0.25, 5, 11).double().cpu()
    want_y, want, want_dx = _formula(block.p, x, dy, mask, block.buckets, grid, H)
    # fp32 throughout, the projections by the library (TF32 off): a few hundred ulps of each
    # tensor's largest value cover sums of a few hundred terms of either sign
    for name, a, b in [("y", y, want_y), ("dx", dx, want_dx)] + [(k, grads[k], want[k]) for k in want]:
        assert (a.double().cpu() - b).abs().max() <= 2e-5 * b.abs().max(), name


def test_training_lowers_the_loss(example):
    losses = example.train(steps=12)
    assert losses[-1] < 0.9 * losses[0] and all(b == b for b in losses)
