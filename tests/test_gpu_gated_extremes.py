"""The gated projections where values are far out: not finite, very large, very unequal."""
import pytest
import torch

import feed_forward_reference as ref

pytestmark = pytest.mark.gpu
TYPES = ["float32", "float16", "bfloat16"]
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid", "identity"]
ORDER = ("dH", "X", "Wg", "Wu", "G", "U")


def _given(rows, D, F, dtype, seed=0, small=1.0):
    """Arguments of the backward call; X and the weights scaled by ``small``."""
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    mk = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(ref.DT[dtype]).cuda()
    W = D ** -0.5 * small
    return dict(dH=mk(rows, F), X=mk(rows, D, std=small), Wg=mk(F, D, std=W), Wu=mk(F, D, std=W),
                G=mk(rows, F), U=mk(rows, F))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("which", ["dH", "G", "U"])
@pytest.mark.parametrize("rows,D,F", [(7, 64, 72), (300, 65, 71)])
def test_gradients_that_are_not_finite_stay_in_their_rows(gs_cuda, rows, D, F, which, value, dtype):
    """dX's other rows, and the other outputs' gradients, have the bits that they have with a 0 in
    that place: among them a row whose dG is beyond fp16's largest number and one of small dG."""
    t = _given(rows, D, F, dtype, 3, 2.0 ** -6)
    row, col = 1, 5
    t["dH"][2], t["U"][2] = t["dH"][2] * 200, t["U"][2] * 600      # |dG| up to 10^6
    t["dH"][3] *= 2.0 ** -10
    t[which][row, col] = 0.0
    want = gs_cuda.gs_gated_linear_backward(**t, bias=True)
    assert all(torch.isfinite(w).all() for w in want[:3])
    ref.check_gated_backward(want, *(t[k] for k in ORDER), "silu", dtype)
    t[which][row, col] = value
    got = gs_cuda.gs_gated_linear_backward(**t, bias=True)
    assert not torch.isfinite(got[0][row]).any()
    for a, b, at in zip(got, want, (row, col, col, col, col)):
        others = torch.arange(a.shape[0], device="cuda") != at
        assert torch.equal(a[others], b[others])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("rows,D,F", [(6, 64, 72), (300, 65, 71)])
def test_a_gradient_of_nothing_costs_other_rows_nothing(gs_cuda, rows, D, F, act, dtype):
    """A row far on the side where the activation and its slope are 0: its dG and dU are zeros, and
    however large its dH and G, the other rows' small gradients keep their bits."""
    t = _given(rows, D, F, dtype, 5)
    t["dH"] *= 2.0 ** -12
    t["G"][0] = -6e4
    t["dH"][0] = 0.0
    want = gs_cuda.gs_gated_linear_backward(**t, activation=act, bias=True)
    ref.check_gated_backward(want, *(t[k] for k in ORDER), act, dtype)
    t["dH"][0] = 6e4
    got = gs_cuda.gs_gated_linear_backward(**t, activation=act, bias=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,D,F", [(48, 64, 72), (300, 65, 71)])
def test_rows_of_very_unequal_gradients(gs_cuda, rows, D, F, act, dtype):
    """dH of one row 2^24 times that of another: each row of dX is off by half steps of its own."""
    t = _given(rows, D, F, dtype, 6, 2.0 ** -4)
    size = 2.0 ** (13 - torch.arange(rows, device="cuda") % 25)
    t["dH"] = (t["dH"].float().clamp(-3, 3) * size[:, None]).to(ref.DT[dtype])
    got = gs_cuda.gs_gated_linear_backward(**t, activation=act, bias=True)
    ref.check_gated_backward(got, *(t[k] for k in ORDER), act, dtype)
