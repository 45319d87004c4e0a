"""gs_gated_linear and its gradient on the GPU against 64-bit formulas."""
import pytest
import torch

import feed_forward_reference as ref

pytestmark = pytest.mark.gpu
TYPES = ["float32", "float16", "bfloat16"]
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid", "identity"]


def _make(rows, D, F, dtype, bias, seed=0):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    mk = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(ref.DT[dtype]).cuda()
    t = dict(X=mk(rows, D), Wg=mk(F, D, std=D ** -0.5), Wu=mk(F, D, std=D ** -0.5),
             bg=mk(F, std=0.5) if bias else None, bu=mk(F, std=0.5) if bias else None)
    return t, mk(rows, F)


def _both(gs, rows, D, F, dtype, act, bias, seed=0):
    t, dH = _make(rows, D, F, dtype, bias, seed)
    H, G, U = gs.gs_gated_linear(**t, activation=act, keep=True)
    ref.check_gated((H, G, U), t["X"], t["Wg"], t["Wu"], t["bg"], t["bu"], act, dtype, "forward")
    assert torch.equal(gs.gs_gated_linear(**t, activation=act), H), "keep changes H"
    back = gs.gs_gated_linear_backward(dH, t["X"], t["Wg"], t["Wu"], G, U, act, bias)
    assert len(back) == (5 if bias else 3)
    ref.check_gated_backward(back, dH, t["X"], t["Wg"], t["Wu"], G, U, act, dtype, "backward")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,D,F", [
    (1, 1, 1), (1, 8, 8), (2, 3, 5), (1, 64, 256), (1, 520, 72), (5, 33, 17), (7, 384, 136),
    (8, 40, 264), (9, 16, 128), (17, 64, 65), (64, 100, 100), (65, 65, 129), (127, 128, 136),
    (128, 72, 128), (129, 257, 40), (255, 64, 130), (256, 128, 256), (257, 192, 264),
    (300, 771, 103), (520, 24, 8), (1000, 1, 3), (513, 136, 640)])
def test_sizes(gs_cuda, rows, D, F, dtype):
    _both(gs_cuda, rows, D, F, dtype, "silu", rows % 2 == 1, rows + D + F)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [1, 3, 140])
def test_activations(gs_cuda, rows, act, dtype):
    _both(gs_cuda, rows, 48, 80, dtype, act, True, 7)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,D,F", [(3000, 192, 520), (2049, 1024, 1160), (40000, 16, 24),
                                      (70001, 9, 8), (100, 64, 3000), (33, 8, 40000)])
def test_larger(gs_cuda, rows, D, F, dtype):
    _both(gs_cuda, rows, D, F, dtype, "gelu_tanh", True, 3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [2, 200])
@pytest.mark.parametrize("which", ["X", "Wg", "Wu", "dH", "G", "all"])
def test_bases_that_are_not_16_byte_aligned(gs_cuda, which, rows, dtype):
    t, dH = _make(rows, 64, 72, dtype, True, 5)
    H, G, U = gs_cuda.gs_gated_linear(**t, keep=True)
    t.update(dH=dH, G=G, U=U)

    def moved(x):
        room = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)
        room[1:] = x.flatten()
        return room[1:].view(x.shape)

    for k in t if which == "all" else [which]:
        t[k] = moved(t[k])
    got = gs_cuda.gs_gated_linear(t["X"], t["Wg"], t["Wu"], t["bg"], t["bu"], keep=True,
                                  out=moved(H) if which == "all" else None)
    ref.check_gated(got, t["X"], t["Wg"], t["Wu"], t["bg"], t["bu"], "silu", dtype)
    back = gs_cuda.gs_gated_linear_backward(t["dH"], t["X"], t["Wg"], t["Wu"], t["G"], t["U"],
                                            bias=True)
    ref.check_gated_backward(back, dH, t["X"], t["Wg"], t["Wu"], G, U, "silu", dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 3, 4, 7, 16, 17, 31, 32])
@pytest.mark.parametrize("D,F", [(40, 4863), (40, 4864), (36, 4867), (131, 5000)])
def test_few_rows_of_many_outputs(gs_cuda, D, F, rows, dtype):
    t, _ = _make(rows, D, F, dtype, True, rows)
    got = gs_cuda.gs_gated_linear(**t, keep=True)
    ref.check_gated(got, t["X"], t["Wg"], t["Wu"], t["bg"], t["bu"], "silu", dtype)


def test_leading_axes_and_views_of_one_projection(gs_cuda):
    t, dH = _make(6, 40, 24, "bfloat16", False)
    packed = torch.cat((t["Wg"], t["Wu"]))
    X = t["X"].view(2, 3, 40)
    H, G, U = gs_cuda.gs_gated_linear(X, packed[:24], packed[24:], keep=True)
    assert H.shape == G.shape == U.shape == (2, 3, 24)
    assert torch.equal(H.view(6, 24), gs_cuda.gs_gated_linear(**t))
    back = gs_cuda.gs_gated_linear_backward(dH.view(2, 3, 24), X, packed[:24], packed[24:], G, U)
    assert back[0].shape == X.shape
    flat = gs_cuda.gs_gated_linear_backward(dH, t["X"], t["Wg"], t["Wu"], G.view(6, 24),
                                            U.view(6, 24))
    for a, b in zip(back, flat):
        assert torch.equal(a.view(b.shape), b)


@pytest.mark.parametrize("dtype", TYPES)
def test_no_rows_and_no_outputs(gs_cuda, dtype):
    for rows, F in ((0, 16), (3, 0), (0, 0)):
        t, dH = _make(rows, 24, F, dtype, True)
        H, G, U = gs_cuda.gs_gated_linear(**t, keep=True)
        assert H.shape == G.shape == U.shape == (rows, F)
        back = gs_cuda.gs_gated_linear_backward(dH, t["X"], t["Wg"], t["Wu"], G, U, bias=True)
        assert [tuple(b.shape) for b in back] == [(rows, 24), (F, 24), (F, 24), (F,), (F,)]
        assert all(not b.any() for b in back)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [3, 150])
def test_large_values_and_rows_that_are_not_finite_stay_in_their_rows(gs_cuda, rows, dtype):
    t, dH = _make(rows, 64, 72, dtype, False, 9)
    clean = gs_cuda.gs_gated_linear(**t)
    t["X"][1, 5] = float("nan")
    got = gs_cuda.gs_gated_linear(**t)
    assert torch.isnan(got[1]).all()
    keep = torch.arange(rows, device="cuda") != 1
    assert torch.equal(got[keep], clean[keep])
    # activations far out: silu and its slope are 0 and 1, no overflow inside
    X = torch.zeros((rows, 8), dtype=ref.DT[dtype], device="cuda")
    X[0, 0], X[1, 0], X[2, 0] = 3e4, -3e4, 1e-6
    Wg = torch.zeros((16, 8), dtype=ref.DT[dtype], device="cuda")
    Wu = Wg.clone()
    Wg[:, 0] = 1
    Wu[:, 1] = 1
    X[:, 1] = 0.5
    for act in ACTS:
        got = gs_cuda.gs_gated_linear(X, Wg, Wu, activation=act, keep=True)
        ref.check_gated(got, X, Wg, Wu, None, None, act, dtype, act)
        d = torch.ones((rows, 16), dtype=ref.DT[dtype], device="cuda")
        back = gs_cuda.gs_gated_linear_backward(d, X, Wg, Wu, got[1], got[2], act)
        ref.check_gated_backward(back[:1], d, X, Wg, Wu, got[1], got[2], act, dtype, act)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 4, 333])
def test_nothing_is_written_outside_and_what_memory_held_does_not_matter(gs_cuda, rows, dtype):
    D, F = 72, 264
    t, dH = _make(rows, D, F, dtype, True, 2)
    want = gs_cuda.gs_gated_linear(**t)
    room = torch.full((rows * F + 64,), 7.0, dtype=ref.DT[dtype], device="cuda")
    n = gs_cuda.gs_gated_linear_workspace_size(rows, D, F, ref.DT[dtype])
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")   # NaN in every type
    out = gs_cuda.gs_gated_linear(**t, out=room[32:32 + rows * F].view(rows, F), workspace=ws)
    assert torch.equal(out, want)
    assert (room[:32] == 7).all() and (room[32 + rows * F:] == 7).all()
    assert (ws[n:] == 255).all()
    _, G, U = gs_cuda.gs_gated_linear(**t, keep=True)
    want = gs_cuda.gs_gated_linear_backward(dH, t["X"], t["Wg"], t["Wu"], G, U, bias=True)
    n = gs_cuda.gs_gated_linear_backward_workspace_size(rows, D, F, ref.DT[dtype])
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    got = gs_cuda.gs_gated_linear_backward(dH, t["X"], t["Wg"], t["Wu"], G, U, bias=True,
                                           workspace=ws)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (ws[n:] == 255).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_repeated_calls_streams_and_graphs_give_the_same_bits(gs_cuda, dtype):
    cases = [_make(rows, 136, 200, dtype, True, rows) for rows in (1, 6, 290)]

    def passes():
        out = []
        for t, dH in cases:
            H, G, U = gs_cuda.gs_gated_linear(**t, keep=True)
            out += [H, G, U] + gs_cuda.gs_gated_linear_backward(dH, t["X"], t["Wg"], t["Wu"], G, U,
                                                                bias=True)
        return out

    want = passes()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(passes())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = passes()
    for _ in range(3):
        for k in kept:
            k.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got.append([k.clone() for k in kept])
    for one in got:
        for a, b in zip(one, want):
            assert torch.equal(a, b)
    assert gs_cuda.gs_device_status() == 0


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(gs_cuda, act):
    t, dH = _make(5, 6, 7, "float32", True, 4)
    t = {k: v.double() for k, v in t.items()}
    f = {k: v.float() for k, v in t.items()}
    _, G, U = gs_cuda.gs_gated_linear(**f, activation=act, keep=True)
    got = gs_cuda.gs_gated_linear_backward(dH, f["X"], f["Wg"], f["Wu"], G, U, act, True)
    loss = lambda: float((ref.gated(t["X"], t["Wg"], t["Wu"], t["bg"], t["bu"], act)[0][0]
                          * dH.double().cpu()).sum())
    step = 1e-5
    for name, grad in zip(("X", "Wg", "Wu", "bg", "bu"), got):
        flat, grad = t[name].view(-1), grad.double().cpu().view(-1)
        for i in range(0, flat.numel(), 3):
            at = flat[i].item()
            flat[i] = at + step
            up = loss()
            flat[i] = at - step
            down = loss()
            flat[i] = at
            # central differences are off by step^2 times a third derivative (under 100 here);
            # the kernel's fp32 gradient by 1e-5 of sums that stay below 50
            assert abs((up - down) / (2 * step) - grad[i]) <= 1e-3, (name, i)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,D,F", [(3, 16, 24), (300, 64, 72), (150, 65, 67)])
@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** 9, 2.0 ** 14])
def test_gradients_of_any_size(gs_cuda, size, rows, D, F, dtype):
    """dH among the type's smallest and near its largest numbers: dG and dU are off by half a
    step, not by a subnormal number's, and stay finite (the results themselves may not be)."""
    t, dH = _make(rows, D, F, dtype, True, 11)
    _, G, U = gs_cuda.gs_gated_linear(**t, keep=True)
    d = (dH.float().clamp(-3, 3) * size).to(ref.DT[dtype])
    small = {k: None if v is None else (v.float() * 2.0 ** -6).to(ref.DT[dtype]) for k, v in t.items()}
    back = gs_cuda.gs_gated_linear_backward(d, small["X"], small["Wg"], small["Wu"], G, U, bias=True)
    ref.check_gated_backward(back, d, small["X"], small["Wg"], small["Wu"], G, U, "silu", dtype)
    zero = torch.zeros_like(dH)
    for b in gs_cuda.gs_gated_linear_backward(zero, t["X"], t["Wg"], t["Wu"], G, U, bias=True):
        assert not b.any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,D,F", [(40, 33000, 24), (3, 40000, 17), (2, 263000, 8)])
def test_wide_rows(gs_cuda, rows, D, F, dtype):
    _both(gs_cuda, rows, D, F, dtype, "silu", True, 6)
