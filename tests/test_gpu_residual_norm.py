"""gs_residual_norm and its gradient on the GPU against 64-bit formulas."""
import pytest
import torch

import feed_forward_reference as ref

pytestmark = pytest.mark.gpu
TYPES = ["float32", "float16", "bfloat16"]
EPS = 1e-5


def _make(rows, D, dtype, post=True, groups=1, biases=True, seed=0, level=0.3):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    mk = lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g) * std + mean).to(
        ref.DT[dtype]).cuda()
    t = dict(X=mk(rows, D, std=1.5, mean=level), Z=mk(rows, D, std=0.8, mean=level),
             Scale=mk(D, std=0.2, mean=1.0), B=mk(D, std=0.2) if biases else None,
             gate=mk(groups, D, std=0.3, mean=0.5) if groups else None,
             z_scale=mk(D, std=0.2, mean=1.0) if post else None,
             z_B=mk(D, std=0.2) if post and biases else None)
    return t, mk(rows, D), mk(rows, D)


def _check(gs, t, dS, dY, dtype, kind="layer", alpha=1.0, eps=EPS):
    D = t["X"].shape[1]
    C = ref.terms(D)
    S, Y, stats = gs.gs_residual_norm(**t, kind=kind, alpha=alpha, epsilon=eps)
    refs, sums = ref.residual_norm(**t, kind=kind, alpha=alpha, eps=eps)
    check_stats = lambda a, r, A: ref.check(a, r, A, "float32", C, what="Stats")
    ref.check(S, refs[0], sums[0], dtype, C, what="S")
    ref.check(Y, refs[1], sums[1], dtype, C, what="Y")
    check_stats(stats, refs[2], sums[2])
    parts = {k: t[k] for k in ("gate", "z_scale", "z_B")}
    back = gs.gs_residual_norm_backward(dS, dY, S, t["Z"], stats, t["Scale"],
                                        bias=t["B"] is not None, kind=kind, alpha=alpha, **parts)
    want = ref.residual_norm_backward(dS, dY, S, t["Z"], stats, t["Scale"], kind=kind, alpha=alpha,
                                      **parts)
    names = {"dX", "dZ", "dScale"} | ({"dB"} if t["B"] is not None else set())
    names |= {"d" + k for k in parts if parts[k] is not None}
    assert set(back) == names
    for k, v in back.items():
        rows = t["X"].shape[0]
        n = D if k in ("dX", "dZ") else D + rows
        ref.check(v, want[k][0], want[k][1], dtype, ref.terms(n), what=k)
    return S, Y, stats, back


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,D", [
    (1, 1), (1, 7), (3, 8), (5, 33), (33, 64), (70, 100), (129, 128), (300, 256), (17, 384),
    (40, 515), (64, 1024), (9, 771), (11, 2048), (7, 2056), (5, 4096), (3, 4104), (3, 6000),
    (2, 8192), (3, 8193), (2, 10000), (2000, 40), (5003, 24)])
def test_sizes(gs_cuda, rows, D, dtype):
    t, dS, dY = _make(rows, D, dtype, seed=rows + D)
    _check(gs_cuda, t, dS, dY, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [20, 43, 61, 90, 127, 170, 250, 333, 500, 701, 1001, 1301, 1999, 2500,
                               4001, 5001, 8191])
def test_widths_of_single_elements(gs_cuda, D, dtype):
    t, dS, dY = _make(38, D, dtype, True, 2, seed=D)
    _check(gs_cuda, t, dS, dY, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [2, 18, 22, 30, 42, 62, 90, 126, 150, 190, 250, 330, 510, 702, 1002, 1302,
                               1998, 2502, 4002, 4102, 5002, 8190, 9002, 20002])
def test_widths_of_pairs(gs_cuda, D, dtype):
    t, dS, dY = _make(38, D, dtype, True, 2, seed=D)
    _check(gs_cuda, t, dS, dY, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [4, 12, 16, 24, 32])
def test_widths_of_few_runs(gs_cuda, D, dtype):
    t, dS, dY = _make(999, D, dtype, True, 3, seed=D)
    _check(gs_cuda, t, dS, dY, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,D", [(30, 64), (30, 520), (5, 8208)])
def test_bases_that_are_aligned_to_pairs(gs_cuda, rows, D, dtype):
    t, dS, dY = _make(rows, D, dtype, seed=9)
    room = torch.empty(rows * D + 2, dtype=ref.DT[dtype], device="cuda")
    room[2:] = t["Z"].flatten()
    _check(gs_cuda, dict(t, Z=room[2:].view(rows, D)), dS, dY, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("post,groups", [(False, 0), (False, 1), (False, 4), (True, 0), (True, 1)])
@pytest.mark.parametrize("D", [4104, 6001, 8192, 8209, 16400, 20001])
def test_forms_of_wide_rows(gs_cuda, D, post, groups, dtype):
    t, dS, dY = _make(20, D, dtype, post, groups, seed=D)
    _check(gs_cuda, t, dS if groups else None, dY, dtype, "rms" if post else "layer")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("biases", [False, True])
@pytest.mark.parametrize("groups", [0, 1, 6, 60])
@pytest.mark.parametrize("D", [48, 77])
def test_forms(gs_cuda, D, groups, biases, post, kind, dtype):
    t, dS, dY = _make(60, D, dtype, post, groups, biases, seed=groups + D)
    _check(gs_cuda, t, dS, dY, dtype, kind, alpha=1.0 if post else -1.75)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,groups,D", [
    (4096, 1, 64), (4096, 4096, 64), (9000, 3000, 40), (6144, 512, 72), (20000, 2500, 16),
    (1500, 500, 1024), (46, 2, 9000), (2100, 700, 8200), (600, 1, 8200)])
def test_gates_of_many_groups(gs_cuda, rows, groups, D, dtype):
    t, dS, dY = _make(rows, D, dtype, True, groups, seed=rows)
    _check(gs_cuda, t, dS, dY, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 520, 8200])
def test_no_gradient_through_the_sum_and_one_gate_for_all(gs_cuda, D, dtype):
    t, dS, dY = _make(50, D, dtype)
    want = _check(gs_cuda, t, None, dY, dtype)[3]
    flat = dict(t, gate=t["gate"][0])
    S, Y, st = gs_cuda.gs_residual_norm(**flat)
    got = gs_cuda.gs_residual_norm_backward(torch.zeros_like(dY), dY, S, t["Z"], st, t["Scale"],
                                            bias=True, gate=flat["gate"], z_scale=t["z_scale"],
                                            z_B=t["z_B"])
    assert got["dgate"].shape == (D,)
    for k in got:
        assert torch.equal(got[k].view(-1), want[k].view(-1)), k


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,D", [(1, 64), (30, 1032), (4, 8208)])
def test_bases_that_are_not_16_byte_aligned(gs_cuda, rows, D, dtype):
    t, dS, dY = _make(rows, D, dtype, seed=8)

    def moved(x):
        room = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)
        room[1:] = x.flatten()
        return room[1:].view(x.shape)

    for k in ("X", "Z", "Scale", "gate", "z_B"):
        _check(gs_cuda, dict(t, **{k: moved(t[k])}), dS, moved(dY) if k == "X" else dY, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_without_variance_and_not_finite(gs_cuda, dtype):
    t, dS, dY = _make(6, 64, dtype, seed=3)
    t["X"][0], t["Z"][0], t["z_B"][:] = 2.0, 0.5, 0.0
    t["gate"][:] = 1.0
    _check(gs_cuda, t, dS, dY, dtype)                      # a constant row: norm 0
    clean = gs_cuda.gs_residual_norm(**t)
    t["Z"][2, 7], t["X"][4, 9] = float("inf"), float("nan")
    got = gs_cuda.gs_residual_norm(**t)
    for a, b in zip(got, clean):
        for r in (0, 1, 3, 5):
            assert torch.equal(a[r], b[r])
    assert torch.isnan(got[1][2]).all() and torch.isnan(got[1][4]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_no_rows_and_no_width(gs_cuda, dtype):
    dt = ref.DT[dtype]
    t, dS, dY = _make(0, 24, dtype, groups=1)
    S, Y, st = gs_cuda.gs_residual_norm(**t)
    assert S.shape == Y.shape == (0, 24) and st.shape == (0, 4)
    back = gs_cuda.gs_residual_norm_backward(dS, dY, S, t["Z"], st, t["Scale"], bias=True,
                                             gate=t["gate"], z_scale=t["z_scale"], z_B=t["z_B"])
    assert all(not v.any() for v in back.values())
    none = torch.empty((3, 0), dtype=dt, device="cuda")
    _, _, st = gs_cuda.gs_residual_norm(none, none, none[0])
    assert torch.isnan(st).all() and st.shape == (3, 4)


@pytest.mark.parametrize("dtype", TYPES)
def test_repeated_calls_streams_graphs_and_workspaces_give_the_same_bits(gs_cuda, dtype):
    cases = [_make(rows, D, dtype, True, groups, seed=D)
             for rows, D, groups in ((1, 64, 1), (96, 520, 8), (700, 24, 1), (12, 8200, 4))]

    def passes(ws=None):
        out = []
        for i, (t, dS, dY) in enumerate(cases):
            S, Y, st = gs_cuda.gs_residual_norm(**t)
            back = gs_cuda.gs_residual_norm_backward(
                dS, dY, S, t["Z"], st, t["Scale"], bias=True, gate=t["gate"], z_scale=t["z_scale"],
                z_B=t["z_B"], workspace=ws[i] if ws else "auto")
            out += [S, Y, st] + [back[k] for k in sorted(back)]
        return out

    want = passes()
    sizes = [gs_cuda.gs_residual_norm_backward_workspace_size(
        t["X"].shape[0], t["X"].shape[1], t["gate"].shape[0], ref.DT[dtype]) for t, _, _ in cases]
    ws = [torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    got = [passes(ws)]
    for w, n in zip(ws, sizes):
        assert (w[n:] == 255).all()
    torch.cuda.synchronize()
    for s in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(s):
            got.append(passes())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = passes()
    for _ in range(2):
        for k in kept:
            k.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got.append([k.clone() for k in kept])
    for one in got:
        for a, b in zip(one, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("post", [False, True])
def test_gradient_against_differences(gs_cuda, post, kind):
    t, dS, dY = _make(6, 9, "float32", post, 2, True, seed=4)
    _, _, _, back = _check(gs_cuda, t, dS, dY, "float32", kind, 1.25)
    w = {k: None if v is None else ref.wide(v) for k, v in t.items()}

    def loss():
        S, Y, _ = ref.residual_norm(**w, kind=kind, alpha=1.25, eps=EPS)[0]
        return float((S * ref.wide(dS)).sum() + (Y * ref.wide(dY)).sum())

    step = 1e-5
    for name, v in w.items():
        if v is None:
            continue
        flat, grad = v.view(-1), ref.wide(back["d" + name]).view(-1)
        for i in range(0, flat.numel(), 2):
            at = flat[i].item()
            flat[i] = at + step
            up = loss()
            flat[i] = at - step
            down = loss()
            flat[i] = at
            # differences are off by step^2 times a third derivative (under 1e4 with deviations
            # near 1); the fp32 gradient by 1e-5 of sums that stay below 100
            assert abs((up - down) / (2 * step) - grad[i]) <= 1e-3, (name, i)
