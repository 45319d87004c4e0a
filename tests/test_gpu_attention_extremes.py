"""Attention under table entries as low (or high) as the types allow: LSE against the 64-bit value,
and gradients that stay finite."""
import math

import pytest
import torch

import block_reference as ref
from block_reference import DT
from test_gpu_attention import DTYPES, Problem, _draw
from spatial_transformer_sampling_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

SATURATED = 3.4028234e38 * math.log(2.0)   # where a base-2 score leaves fp32's range


def _problem(gs, seed, dtype, entry, Lq=80, Lk=80, D=64, share=False):
    """Every pair of one bucket, or (`share`) the keys after the query in it and the others in
    another of ordinary entries."""
    off = torch.arange(Lq + Lk - 1) - (Lk - 1)
    buckets = torch.where(off < 0, 0, 1 if share else 0).to(torch.int32)
    table = _draw(wl.rng(seed), (2, 1), dtype)
    table[0] = entry
    return Problem(gs, seed, dtype, 1, 1, D, (1, Lq), (1, Lk), table=table, buckets=buckets)


def _entries(names):
    """(dtype, entry) for the entries that the type holds."""
    out = []
    for dtype in DTYPES:
        low = torch.finfo(DT[dtype]).min
        for name in names:
            entry = {"lowest": low, "highest": -low}.get(name, name)
            if abs(entry) <= -low:
                out.append((dtype, entry))
    return out


SHAPES = [(80, 80, 64), (80, 80, 20), (3, 80, 64), (40, 1500, 64), (40, 1500, 20)]


@pytest.mark.parametrize("Lq,Lk,D", SHAPES)
@pytest.mark.parametrize("dtype,entry", _entries(["lowest", "highest", -1e38, -1e20, -1e9, 1e9, -6e4,
                                                  -1e4]))
def test_lse_of_rows_of_one_extreme_entry(gs_cuda, entry, Lq, Lk, D, dtype):
    p = _problem(gs_cuda, 700, dtype, entry, Lq, Lk, D)
    bias = p.bias.clamp(-SATURATED, SATURATED)
    _, lse, _ = ref.attention(p.Q, p.K, p.V, p.scale, bias)
    O, LSE = gs_cuda.gs_attention(*p.qkv(), **p.args())
    assert torch.isfinite(O).all()
    # the entry times log2 e, the score's sum with it, the logarithm's and the way back: four
    # roundings of numbers of LSE's size, and two steps of it at the most
    err = (LSE.double().cpu() - lse).abs()
    assert (err <= 6 * 2.0 ** -23 * lse.abs() + 256 * 2.0 ** -24).all(), (err / lse.abs()).max()


@pytest.mark.parametrize("Lq,Lk,D", SHAPES)
@pytest.mark.parametrize("dtype,entry", _entries(["lowest", "highest", -1e38, -1e20, -1e9, 1e9, -1e7,
                                                  -6e4, -1e4]))
def test_gradients_of_rows_of_one_extreme_entry_stay_finite(gs_cuda, entry, Lq, Lk, D, dtype):
    p = _problem(gs_cuda, 710, dtype, entry, Lq, Lk, D)
    Q, K, V = p.qkv()
    O, LSE = gs_cuda.gs_attention(Q, K, V, **p.args())
    given = [LSE]
    if abs(entry) >= 1e20:   # the entry itself, as other code would round the 64-bit value
        given.append(torch.full_like(LSE, _draw(wl.rng(0), (1,), dtype).fill_(entry).item()))
    dO = p.dO.cuda()
    for lse in given:
        dQ, dK, dV, dT = gs_cuda.gs_attention_backward(dO, Q, K, V, O, lse, **p.args())
        for name, t in (("dQ", dQ), ("dK", dK), ("dV", dV), ("dTable", dT)):
            assert torch.isfinite(t.float()).all(), name
        do, v, k = (t.double().cpu() for t in (p.dO, p.V, p.K))
        # no weight is above 1 (by more than a step of LSE below 2^20)
        most = math.exp(2.0 ** -3) if abs(entry) < 1e9 else 1.0 + 2.0 ** -7
        lim = most * do.abs().sum(1, keepdim=True) * 1.01 + 1e-3
        assert (dV.double().cpu().abs() <= lim).all()
        if abs(entry) >= 1e20:   # scores and LSE are the entry: the weights are 1
            want = do.sum(1, keepdim=True).expand_as(dV)
            ref.check(dV, want, do.abs().sum(1, keepdim=True).expand_as(dV), dtype, "dV")


@pytest.mark.parametrize("dtype,entry", _entries(["lowest", -1e38, -1e9, -6e4]))
@pytest.mark.parametrize("D", [64, 20])
def test_gradients_beside_lowest_entries_are_those_of_masked_pairs(gs_cuda, D, entry, dtype):
    p = _problem(gs_cuda, 720, dtype, entry, D=D, share=True)
    p.both()
    got = p.backward()
    p.table[0] = float("-inf")
    p.bias, p.which = ref.pair_bias(p.table, p.buckets, p.q, p.k)
    for a, b in zip(got, p.backward()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("Lq,Lk,D", SHAPES)
@pytest.mark.parametrize("entry", [-3e9, 3e9, -1e10])
def test_scores_of_several_steps_of_an_extreme_lse(gs_cuda, entry, Lq, Lk, D, dtype):
    # scores of millions beside an entry whose spacing is up to a thousand: LSE must not end up a step
    # below a row's largest score, whose weight would be 2^256 and more
    p = _problem(gs_cuda, 730, dtype, entry, Lq, Lk, D)
    p.Q = (p.Q.float() * 4e6).to(p.Q.dtype)
    Q, K, V = p.qkv()
    O, LSE = gs_cuda.gs_attention(Q, K, V, **p.args())
    dQ, dK, dV, dT = gs_cuda.gs_attention_backward(p.dO.cuda(), Q, K, V, O, LSE, **p.args())
    assert all(torch.isfinite(t.float()).all() for t in (O, LSE, dQ, dK, dV, dT))
    do = p.dO.double()
    lim = (1.0 + 2.0 ** -7) * do.abs().sum(1, keepdim=True) * 1.01 + 1e-3
    assert (dV.double().cpu().abs() <= lim).all()
