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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [5, 200])
def test_projections_as_large_as_the_type_holds(gs_cuda, rows, act, dtype):
    """H is finite where act(G) U is, and the slopes far out are 0, 1 or the factor's own."""
    dt = ref.DT[dtype]
    far = [1e4, 65504.0] if dtype == "float16" else [3e4, 1e18, 1e20, 3e30, 3e38]
    far = torch.tensor(far + [-v for v in far])
    small = 2.0 ** -10 if dtype == "float16" else 2.0 ** -100
    X = torch.zeros((rows, 8))
    X[:, 0], X[:, 1] = far.repeat(-(-rows // len(far)))[:rows], small
    W = torch.zeros((2, 16, 8))
    W[0, :, 0] = W[1, :, 1] = 1.0
    X, Wg, Wu = X.to(dt).cuda(), W[0].to(dt).cuda(), W[1].to(dt).cuda()
    got = gs_cuda.gs_gated_linear(X, Wg, Wu, activation=act, keep=True)
    ref.check_gated(got, X, Wg, Wu, None, None, act, dtype, act)
    dH = torch.full((rows, 16), small, dtype=dt, device="cuda")
    U = torch.ones_like(dH)
    back = gs_cuda.gs_gated_linear_backward(dH, X, Wg, Wu, got[1], U, act, True)
    ref.check_gated_backward(back[:1], dH, X, Wg, Wu, got[1], U, act, dtype, act)
    # the biases' sums by themselves: a row at a time
    for r in range(min(rows, len(far))):
        one = [t[r:r + 1].contiguous() for t in (dH, X, got[1], U)]
        back = gs_cuda.gs_gated_linear_backward(one[0], one[1], Wg, Wu, one[2], one[3], act, True)
        _, slope = ref.act(act, ref.wide(one[2]))
        ref.check(back[3], (ref.wide(one[0]) * slope)[0], (ref.wide(one[0]) * (slope.abs() + 1))[0],
                  dtype, 64, what="dbg")
