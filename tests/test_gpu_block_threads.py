"""First calls of the transformer-block operators from several host threads at once: the kernels'
per-device setup (shared-memory limits, cluster sizes, tensor-map encoder) is the library's only
state.  A fresh process starts eight threads that make their first calls together, each on its own
stream; every result is compared with the same call made alone, and with the 64-bit reference."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import sys, threading
import torch
sys.path.insert(0, sys.argv[1])
sys.path.insert(0, sys.argv[1] + "/tests")
import block_reference as ref
import spatial_transformer_sampling_gb300 as gs

gs.load_library()
dev = torch.device("cuda:0")
torch.cuda.set_device(dev)
T = 8
DT = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
# N, H, D, queries, keys: few queries alone and over a cluster, one block per 128 queries, blocks
# of several short heads, keys shared by a cluster, wide heads, widths that are not 16 bytes
SHAPES = [(2, 2, 64, (1, 1), (1, 1500)), (1, 2, 64, (2, 3), (1, 90)), (6, 60, 64, (9, 16), (9, 16)),
          (130, 3, 32, (6, 6), (6, 6)), (1, 2, 64, (1, 40), (1, 1100)), (2, 2, 128, (8, 20), (8, 20)),
          (2, 2, 20, (5, 17), (5, 17))]
maps = [gs.gs_relative_buckets(q, k, 8, 32, device="cpu") for _, _, _, q, k in SHAPES]


def inputs(t):
    g = torch.Generator()
    g.manual_seed(100 + t)
    mk = lambda *s: torch.randn(s, generator=g)
    cases = []
    for (N, H, D, q, k), (m, rows) in zip(SHAPES, maps):
        for dt in DT.values():
            cases.append([x.to(dt) for x in (mk(N, q[0] * q[1], H, D), mk(N, k[0] * k[1], H, D),
                                             mk(N, k[0] * k[1], H, D), mk(N, q[0] * q[1], H, D),
                                             mk(rows, H))] + [m, q, k])
    norms = [[x.to(dt) for x in (mk(50, D), mk(D), mk(50, D))] for dt in DT.values()
             for D in (64, 1024, 771, 9000)]
    return cases, norms


def calls(cases, norms):
    out = []
    for Q, K, V, dO, table, m, q, k in cases:
        O, LSE = gs.gs_attention(Q, K, V, table, m, q, k)
        out += [O, LSE, gs.gs_attention(Q, K, V)[0]]
        out += gs.gs_attention_backward(dO, Q, K, V, O, LSE, table, m, q, k)
    for X, S, dY in norms:
        Y, M, I = gs.gs_layer_norm(X, S)
        out += [Y, M, I, *gs.gs_layer_norm_backward(dY, X, S, M, I)]
        out += [gs.gs_dropout(X, 0.3, 5, 6), gs.gs_dropout(X, 0.3, 5, 6, residual=Y)]
    return out


dev_of = lambda lists: [[x.to(dev) if torch.is_tensor(x) else x for x in row] for row in lists]
given = [inputs(t) for t in range(T)]
results, start = [None] * T, threading.Barrier(T)


def work(t):
    cases, norms = (dev_of(x) for x in given[t])
    s = torch.cuda.Stream(dev)
    torch.cuda.synchronize(dev)
    start.wait()
    with torch.cuda.stream(s):
        r = calls(cases, norms)
    s.synchronize()
    results[t] = r


threads = [threading.Thread(target=work, args=(t,)) for t in range(T)]
for th in threads: th.start()
for th in threads: th.join()
assert gs.gs_device_status() == 0
for t in range(T):
    again = calls(*(dev_of(x) for x in given[t]))
    assert results[t] is not None and len(again) == len(results[t])
    for i, (a, b) in enumerate(zip(results[t], again)):
        assert torch.equal(a, b), (t, i)
# and what they agree on is right
at = 0
for (N, H, D, q, k), (m, rows) in zip(SHAPES, maps):
    for name in DT:
        Q, K, V, dO, table, _, _, _ = given[0][0][at]
        bias, _ = ref.pair_bias(table, m, q, k)
        o, lse, A = ref.attention(Q, K, V, D ** -0.5, bias)
        ref.check(results[0][7 * at], o, A, name, str(q))
        at += 1
print("threads ok")
"""


def test_first_calls_from_eight_host_threads(gs_cuda):
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT], capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
