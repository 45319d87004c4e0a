"""The example's feed-forward half on the GPU: the operators together, as they are used, against
64-bit automatic differentiation of the same formulas."""
import importlib.util
import os
import sys

import pytest
import torch

import feed_forward_reference as ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "glimpse_feed_forward.py")


@pytest.fixture(scope="module")
def example(gs_cuda):
    spec = importlib.util.spec_from_file_location("glimpse_feed_forward", PATH)
    module = importlib.util.module_from_spec(spec)
    sys.modules["glimpse_feed_forward"] = module
    spec.loader.exec_module(module)
    return module


def _formula(p, x, c, dy, ds, activation, eps=1e-5):
    """Outputs and gradients of sum(y dy) + sum(s ds) in 64 bits by automatic differentiation."""
    leaf = {k: v.detach().double().cpu().requires_grad_(True) for k, v in p.items()}
    x = x.detach().double().cpu().requires_grad_(True)

    def norm(t, g, b):
        d = t - t.mean(2, keepdim=True)
        return d / torch.sqrt((d * d).mean(2, keepdim=True) + eps) * g + b

    u = norm(x, leaf["g0"], leaf["b0"])
    g, v = u @ leaf["Wg"].t() + leaf["bg"], u @ leaf["Wu"].t() + leaf["bu"]
    z = (ref.act(activation, g)[0] * v) @ leaf["Wd"].t()
    gate = (c.double().cpu() @ leaf["Wc"]).unsqueeze(1)
    s = x + gate * norm(z, leaf["gz"], leaf["bz"])
    y = norm(s, leaf["g1"], leaf["b1"])
    ((y * dy.double().cpu()).sum() + (s * ds.double().cpu()).sum()).backward()
    return y.detach(), {k: t.grad for k, t in leaf.items()}, x.grad


@pytest.mark.parametrize("activation", ["silu", "gelu"])
@pytest.mark.parametrize("N,L,C,hidden", [(3, 42, 32, 88), (2, 150, 65, 131), (1, 1, 48, 64)])
def test_gradients_match_automatic_differentiation(example, gs_cuda, N, L, C, hidden, activation):
    block = example.FeedForward(C, hidden, 5, torch.float32, activation, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda")
    for name in ("g0", "b0", "gz", "bz", "g1", "b1"):
        block.p[name] = block.p[name] + 0.1 * mk(C)
    x, c, dy, ds = mk(N, L, C), mk(N, 5), mk(N, L, C), mk(N, L, C)
    y = block.forward(x, c)
    grads, dx = block.backward(dy, ds)
    want_y, want, want_dx = _formula(block.p, x, c, dy, ds, activation)
    assert set(grads) == set(want)
    # fp32 throughout, the plain products by the library (TF32 off): a few hundred ulps of each
    # tensor's largest value cover sums of a few hundred terms of either sign through three norms
    for name, a, b in [("y", y, want_y), ("dx", dx, want_dx)] + [(k, grads[k], want[k]) for k in want]:
        assert (a.double().cpu() - b).abs().max() <= 3e-5 * b.abs().max(), name


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_training_runs_in_16_bits(example, gs_cuda, dtype):
    losses = example.train(steps=3, N=2, grid=(5, 6), dtype=ref.DT[dtype])
    assert len(losses) == 3 and all(v == v and v != float("inf") for v in losses)
    assert gs_cuda.gs_device_status() == 0


def test_a_training_step_in_a_graph_gives_the_same_bits(example, gs_cuda):
    block = example.FeedForward(40, 72, 4, torch.bfloat16)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    x, c, dy = mk(2, 70, 40), mk(2, 4), mk(2, 70, 40)

    def step():
        y = block.forward(x, c)
        grads, dx = block.backward(dy)
        return [y, dx] + [grads[k] for k in sorted(grads)]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):   # the library products' own workspaces, outside the capture
        step()
    torch.cuda.synchronize()
    want = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for fill in (0.0, 1.0):
        for t in kept:
            t.fill_(fill)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(a, b)
