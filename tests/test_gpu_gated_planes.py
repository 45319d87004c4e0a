"""The gated projections' fp32 products, positive throughout, to a few steps of their results: every
product of planes, in every run, operand and part, on its own account."""
import pytest
import torch

import gated_planes as gp

pytestmark = pytest.mark.gpu


def _runs(K, operands=1):
    return operands * -(-K // (gp.RUN * gp.STAGE))


@pytest.mark.parametrize("rows,F", [(40, 40), (200, 264), (577, 1031)])
@pytest.mark.parametrize("D", [40, 256, 300, 512, 1024, 2048])
def test_projections(gs_cuda, D, rows, F):
    X, Wg, Wu = (gp.planed(n, D, seed=D + i) for i, n in enumerate((rows, F, F)))
    _, G, U = gs_cuda.gs_gated_linear(X.cuda(), Wg.cuda(), Wu.cuda(), activation="identity", keep=True)
    assert gp.off(G, gp.exact([(X, Wg)])) <= gp.bound(_runs(D))
    assert gp.off(U, gp.exact([(X, Wu)])) <= gp.bound(_runs(D))


# `parts`: that a contraction is shared out into, whose sums are added as the runs' are
@pytest.mark.parametrize("rows,D,F,parts", [
    (300, 72, 256, 0), (512, 40, 300, 0), (1024, 264, 512, 2), (300, 771, 1024, 4), (2048, 136, 72, 4),
    (4096, 40, 24, 8), (64, 40, 4096, 16)])
def test_gradients(gs_cuda, rows, D, F, parts):
    """identity with U = 1 and G = 2: dG = dH and dU = 2 dH."""
    dH, X = gp.planed(rows, F, seed=1), gp.planed(rows, D, seed=2)
    Wg, Wu = gp.planed(F, D, seed=3), gp.planed(F, D, seed=4)
    one = torch.ones((rows, F), device="cuda")
    dX, dWg, dWu = gs_cuda.gs_gated_linear_backward(dH.cuda(), X.cuda(), Wg.cuda(), Wu.cuda(), 2 * one,
                                                    one, activation="identity")
    want = gp.exact([(dH, Wg.T), (2 * dH, Wu.T)])
    assert gp.off(dX, want) <= gp.bound(_runs(F, 2) + parts)
    want = gp.exact([(dH.T, X.T)])
    assert gp.off(dWg, want) <= gp.bound(_runs(rows) + parts)
    assert gp.off(dWu, 2 * want) <= gp.bound(_runs(rows) + parts)
