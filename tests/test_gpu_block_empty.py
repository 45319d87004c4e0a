"""Calls of the transformer-block operators whose extents hold no element."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_layer_norm_statistics_of_no_element_are_nan(gs_cuda):
    X, S = torch.empty((5, 0), device="cuda"), torch.empty(0, device="cuda")
    held = [torch.full((5, 1), 7.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    held.clear()             # what the allocator hands out next holds numbers
    Y, M, I = gs_cuda.gs_layer_norm(X, S)
    assert Y.shape == (5, 0) and M.shape == (5, 1)
    assert torch.isnan(M).all() and torch.isnan(I).all()
    dX, dS, dB = gs_cuda.gs_layer_norm_backward(X, X, S, M, I)
    assert dX.shape == (5, 0) and dS.shape == (0,) and dB.shape == (0,)
