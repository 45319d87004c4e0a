"""First calls of the feed-forward operators in a fresh process: from several host threads at once,
each on its own stream, and inside the capture of a graph.  Every result is compared with the same
call made alone, and the first with the 64-bit reference."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = r"""
import sys, threading
import torch
sys.path.insert(0, sys.argv[1])
sys.path.insert(0, sys.argv[1] + "/tests")
import feed_forward_reference as ref
import spatial_transformer_sampling_gb300 as gs

gs.load_library()
dev = torch.device("cuda:0")
torch.cuda.set_device(dev)
# few rows, one pair of CTAs, narrow and wide tiles, odd widths, a shared contraction
GATED = [(3, 64, 72), (200, 64, 40), (300, 65, 67), (3000, 40, 24), (700, 520, 1096)]
# a team per row from 8 lanes to a block, staged rows, wide ones; rows, D, groups
NORM = [(40, 24, 1), (60, 77, 6), (64, 520, 4), (33, 1024, 0), (5, 6000, 1), (4, 9000, 2)]


def inputs(t):
    g = torch.Generator()
    g.manual_seed(100 + t)
    mk = lambda *s: torch.randn(s, generator=g)
    gated = [[x.to(dt) for x in (mk(r, D), mk(F, D) * D ** -0.5, mk(F, D) * D ** -0.5, mk(F), mk(F),
                                 mk(r, F))] for r, D, F in GATED for dt in ref.DT.values()]
    norm = [[x.to(dt) for x in (mk(r, D), mk(r, D), mk(D), mk(D), mk(max(n, 1), D), mk(r, D), mk(r, D))]
            + [n] for r, D, n in NORM for dt in ref.DT.values()]
    return gated, norm


def calls(gated, norm):
    out = []
    for X, Wg, Wu, bg, bu, dH in gated:
        H, G, U = gs.gs_gated_linear(X, Wg, Wu, bg, bu, keep=True)
        out += [H, G, U, gs.gs_gated_linear(X, Wg, Wu, activation="gelu")]
        out += gs.gs_gated_linear_backward(dH, X, Wg, Wu, G, U, bias=True)
    for X, Z, a, b, gate, dS, dY, n in norm:
        form = dict(gate=gate if n else None, z_scale=a, z_B=b)
        S, Y, st = gs.gs_residual_norm(X, Z, a, b, **form)
        back = gs.gs_residual_norm_backward(dS, dY, S, Z, st, a, bias=True, **form)
        out += [S, Y, st] + [back[k] for k in sorted(back)]
        S, Y, st = gs.gs_residual_norm(X, Z, a, kind="rms")
        back = gs.gs_residual_norm_backward(None, dY, S, Z, st, a, kind="rms")
        out += [S, Y, st] + [back[k] for k in sorted(back)]
    return out


on_device = lambda lists: [[x.to(dev) if torch.is_tensor(x) else x for x in row] for row in lists]


def check_first(results, given):
    X, Wg, Wu, bg, bu, dH = given[0][0]
    ref.check_gated(results[:3], X, Wg, Wu, bg, bu, "silu", "float32")
    ref.check_gated_backward(results[4:9], dH, X, Wg, Wu, results[1], results[2], "silu", "float32")
"""

THREADS = COMMON + r"""
T = 8
given = [inputs(t) for t in range(T)]
results, start = [None] * T, threading.Barrier(T)


def work(t):
    gated, norm = (on_device(x) for x in given[t])
    s = torch.cuda.Stream(dev)
    torch.cuda.synchronize(dev)
    start.wait()
    with torch.cuda.stream(s):
        r = calls(gated, norm)
    s.synchronize()
    results[t] = r


threads = [threading.Thread(target=work, args=(t,)) for t in range(T)]
for th in threads: th.start()
for th in threads: th.join()
assert gs.gs_device_status() == 0
for t in range(T):
    again = calls(*(on_device(x) for x in given[t]))
    assert results[t] is not None and len(again) == len(results[t])
    for i, (a, b) in enumerate(zip(results[t], again)):
        assert torch.equal(a, b), (t, i)
check_first(results[0], given[0])
print("threads ok")
"""

CAPTURE = COMMON + r"""
given = inputs(0)
gated, norm = (on_device(x) for x in given)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    kept = calls(gated, norm)
graph.replay()
torch.cuda.synchronize()
first = [k.clone() for k in kept]
check_first(first, given)
# a second graph of the same calls has workspaces of its own; replayed on two streams at once
other = torch.cuda.CUDAGraph()
with torch.cuda.graph(other):
    kept2 = calls(gated, norm)
a, b = torch.cuda.Stream(), torch.cuda.Stream()
for _ in range(5):
    with torch.cuda.stream(a): graph.replay()
    with torch.cuda.stream(b): other.replay()
torch.cuda.synchronize()
again = calls(gated, norm)
for i, (x, y, z, w) in enumerate(zip(first, kept, kept2, again)):
    assert torch.equal(x, y) and torch.equal(x, z) and torch.equal(x, w), i
assert gs.gs_device_status() == 0
print("capture ok")
"""


@pytest.mark.parametrize("name,script", [("threads", THREADS), ("capture", CAPTURE)],
                         ids=["threads", "capture"])
def test_first_calls(gs_cuda, name, script):
    r = subprocess.run([sys.executable, "-c", script, ROOT], capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and f"{name} ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
