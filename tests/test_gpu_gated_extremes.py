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


def _phi(g):
    """By erfc: torch.special.ndtr loses its digits below -5 as 1 + erf does (at -8 it is 2 % off)."""
    return 0.5 * torch.erfc(-g * 0.5 ** 0.5)


def _phi_off(g, dtype):
    """How far Phi(g) and e^(-g^2/2) may be off, relative to them, in steps of 2^-24: the argument of
    the exponential is formed of three factors rounded by half a step each, which move it by up to
    3 half steps of its g^2 / 2; 32 for the functions (up to 2 ulps each) and the formula around
    them.  In 16-bit types Phi comes of a polynomial that is off by 1.1e-6 of it at most."""
    return 1.5 * g * g + 32 + (0 if dtype == "float32" else 1.1e-6 * 2.0 ** 24)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,aligned", [(1, True), (24, True), (300, True), (300, False)])
def test_gelu_keeps_its_digits_where_it_is_small(gs_cuda, rows, aligned, dtype):
    """G = g and U = 2^12 exactly: H is off by half a step of itself, however small Phi(g) is."""
    dt, F = ref.DT[dtype], 40
    X = torch.zeros((rows, 8))
    g = torch.linspace(-6.0 if dtype == "float16" else -8.0, 3.0, rows * F).to(dt)
    # a row has one G in all columns or, by the weights, F of them
    X[:, 0], X[:, 1] = (g.view(rows, F)[:, 0].float() if rows > 1 else 1.0), 1.0
    Wg, Wu = torch.zeros((F, 8)), torch.zeros((F, 8))
    Wg[:, 0] = 1.0 if rows > 1 else g.float()
    Wu[:, 1] = 2.0 ** 12

    def moved(t):   # a base that starts on no 16-byte boundary
        room = torch.empty(t.numel() + 8, dtype=dt, device="cuda")
        at = room[0 if aligned else 1:][:t.numel()].view(t.shape)
        return at.copy_(t)

    X, Wg, Wu = moved(X), moved(Wg), moved(Wu)
    H, G, U = gs_cuda.gs_gated_linear(X, Wg, Wu, activation="gelu", keep=True)
    exact = ref.wide(X)[:, :1] * ref.wide(Wg)[:, 0]
    assert torch.equal(ref.wide(G), exact)
    want = exact * _phi(exact) * 2.0 ** 12
    ref.check(H, want, want.abs(), dtype, _phi_off(exact, dtype), what="H")


@pytest.mark.parametrize("dtype", TYPES)
def test_gelu_gradients_keep_their_digits_where_they_are_small(gs_cuda, dtype):
    """The biases' gradients of a single row are dU and dG themselves."""
    dt, F = ref.DT[dtype], 4000
    g = torch.linspace(-6.0 if dtype == "float16" else -8.0, 3.0, F).to(dt).cuda()[None]
    t = _given(1, 8, F, dtype, 2)
    t.update(G=g, U=torch.full_like(g, 2.0 ** 6), dH=torch.full_like(g, 2.0 ** 6))
    got = gs_cuda.gs_gated_linear_backward(**t, activation="gelu", bias=True)
    g = ref.wide(g)[0]
    density = torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5
    a, slope = g * _phi(g), _phi(g) + g * density
    off = _phi_off(g, dtype)
    ref.check(got[4], a * 64, a.abs() * 64, dtype, off, what="dU")
    ref.check(got[3], slope * 4096, (_phi(g) + g.abs() * density) * 4096, dtype, off,
              what="dG")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_rows_that_no_copy_serves_are_not_copied(gs_cuda, dtype):
    """Forward rows beyond 32768 elements are read where they lie: the workspace stays as it was."""
    rows, D, F = 40, 32777, 24
    t = _given(rows, D, F, dtype, 8)
    t = {k: t[k] for k in ("X", "Wg", "Wu")}
    n = gs_cuda.gs_gated_linear_workspace_size(rows, D, F, ref.DT[dtype])
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")
    got = gs_cuda.gs_gated_linear(**t, keep=True, workspace=ws)
    ref.check_gated(got, t["X"], t["Wg"], t["Wu"], None, None, "silu", dtype)
    assert (ws == 255).all()
