"""Attention's gradient over the range of magnitudes that the types hold: the bounds are those of
block_reference.py, whatever dO's and V's scale."""
import pytest
import torch

import block_reference as ref
from block_reference import DT
from test_gpu_attention import Problem

pytestmark = pytest.mark.gpu


def _scaled(t, factor):
    return (t.float() * factor).to(t.dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("size", [1e-4, 1e-3, 1.0, 1e3])
@pytest.mark.parametrize("bias", [True, False])
def test_gradients_small_and_large_over_many_keys(gs_cuda, bias, size, dtype):
    # weights of about 2^-11: the rounded gradient of a score has to keep its precision
    p = Problem(gs_cuda, 600, dtype, 1, 1, 64, (1, 2048), (1, 2048), 32, bias=bias)
    p.dO = _scaled(p.dO, size)
    p.backward()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("D", [64, 128])
def test_gradients_of_a_scaled_loss_over_short_heads(gs_cuda, D, dtype):
    # dO . v beyond fp16's range, the gradients themselves inside it but for a few entries of the
    # table's, whose sums over the batch and eight queries are infinite in the type
    p = Problem(gs_cuda, 610, dtype, 2, 2, D, (8, 8), (8, 8), 0)
    p.dO = _scaled(p.dO, 1.2e4)
    o, lse, _ = ref.attention(p.Q, p.K, p.V, p.scale, p.bias)
    O, LSE = o.to(DT[dtype]).contiguous(), lse.float()
    grads, sums = ref.attention_backward(p.dO, p.Q, p.K, p.V, O, LSE, p.scale, p.bias, None, p.which,
                                         p.table.shape[0])
    most = torch.finfo(DT[dtype]).max
    assert all(g.abs().max() < most for g in grads[:3])
    got = gs_cuda.gs_attention_backward(p.dO.cuda(), *p.qkv(), O.cuda(), LSE.cuda(), **p.args())
    for name, a, r, A in zip(("dQ", "dK", "dV", "dTable"), got, grads, sums):
        lim = ref.bound(r, A, dtype)
        beyond = r.abs() - lim > most
        r = torch.where(beyond, r.sign() * float("inf"), r)
        doubt = ~beyond & (r.abs() + lim > most)   # may be infinite or not
        ref.check(a, torch.where(doubt, a.double().cpu(), r), A, dtype, name)


@pytest.mark.parametrize("L", [9, 12])
def test_score_gradients_beyond_the_type_with_gradients_inside_it(gs_cuda, L):
    p = Problem(gs_cuda, 640, "float16", 8, 4, 128, (1, L), (1, L), bias=False)
    p.dO = _scaled(p.dO, 1.2e4)
    o, lse, _ = ref.attention(p.Q, p.K, p.V, p.scale)
    q, k, v, do, o = (t.double().permute(0, 2, 1, 3) for t in (p.Q, p.K, p.V, p.dO, o.half()))
    w = torch.exp(q @ k.transpose(2, 3) * p.scale - lse.unsqueeze(3))
    ds = w * (do @ v.transpose(2, 3) - (do * o).sum(3, keepdim=True))
    assert ds.abs().max() > 1.05 * torch.finfo(torch.float16).max
    assert all(torch.isfinite(g).all() for g in p.backward())


@pytest.mark.parametrize("by_key,by_query", [(1e-3, 1e3), (2e3, 1e-3), (1e-5, 1e-2)])
def test_gradients_where_values_and_dO_differ_in_size(gs_cuda, by_key, by_query):
    p = Problem(gs_cuda, 620, "float16", 2, 2, 40, (12, 20), (12, 20), 8, k_len=[240, 100])
    p.V, p.dO = _scaled(p.V, by_key), _scaled(p.dO, by_query)
    p.backward()


def test_a_row_that_is_not_finite_changes_no_other_rows_scale(gs_cuda):
    p = Problem(gs_cuda, 630, "float16", 1, 2, 64, (1, 300), (1, 300), 16)
    p.dO = _scaled(p.dO, 1e-4)
    dQ = p.backward()[0]
    o, lse, _ = ref.attention(p.Q, p.K, p.V, p.scale, p.bias)
    p.dO[0, 5, 0, 3], p.dO[0, 7, 1, 0] = float("inf"), float("nan")
    got = p.gs.gs_attention_backward(p.dO.cuda(), *p.qkv(), o.to(DT["float16"]).contiguous().cuda(),
                                     lse.float().cuda(), **p.args())[0]
    keep = torch.tensor([i for i in range(300) if i not in (5, 7)], device="cuda")
    assert not torch.isfinite(got[0, 5, 0]).any() and not torch.isfinite(got[0, 7, 1]).any()
    # the scale may come from another row, a power of two away: both round what they hold
    a, b = got[0, keep].double(), dQ[0, keep].double()
    assert ((a - b).abs() <= 2.0 ** -9 * b.abs().amax() + 2.0 ** -23).all()
