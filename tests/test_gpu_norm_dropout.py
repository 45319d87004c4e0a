"""Layer norm and dropout on the GPU against 64-bit references (block_reference.py holds the
references and the derivation of the bounds)."""
import numpy as np
import pytest
import torch

import block_reference as ref
from block_reference import DT
from spatial_transformer_sampling_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "float16", "bfloat16"]
# widths around vector, warp and block sizes, odd ones, and beyond what a row keeps on chip
NORM_SHAPES = [(1, 1), (1, 64), (3, 7), (5, 33), (64, 64), (1000, 48), (257, 127), (9, 255),
               (33, 771), (130, 1024), (17, 1025), (6, 4096), (3, 5000), (5, 8192), (2, 8193),
               (2, 20011)]


def _norm_inputs(seed, rows, D, dtype, level=1.0):
    g = wl.rng(seed)
    x = g.normal(size=(rows, D)) * 1.5 + level * g.normal(size=(rows, 1))
    make = lambda a: wl.as_dtype(a, dtype)
    return (make(x), make(1.0 + 0.2 * g.normal(size=D)), make(0.2 * g.normal(size=D)),
            make(g.normal(size=(rows, D))))


def _norm_terms(x, scale, b, mean, inv):
    """Sum of absolute terms of Y: the mean is off by ulps of mean |x|, which the row's level
    may make larger than x - mean."""
    level = x.abs().mean(1, keepdim=True) + x.abs()
    return (level * inv * scale.abs()) + (b.abs() if b is not None else 0.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,D", NORM_SHAPES)
def test_layer_norm_and_gradient(gs_cuda, rows, D, dtype):
    X, S, B, dY = _norm_inputs(7 * rows + D, rows, D, dtype)
    x, s, b, dy = (t.double() for t in (X, S, B, dY))
    y, mean, inv = ref.layer_norm(x, s, b, 1e-5)
    Xd, Sd, Bd, dYd = X.cuda(), S.cuda(), B.cuda(), dY.cuda()
    Y, M, I = gs_cuda.gs_layer_norm(Xd, Sd, Bd)
    # D = 1: x - mean is 0 exactly; elsewhere the statistics are sums of D fp32 terms
    ref.check(M, mean, x.abs().mean(1, keepdim=True), "float32", "mean")
    ref.check(I, inv, inv * (1 + x.abs().mean(1, keepdim=True) * inv), "float32", "inv")
    terms = _norm_terms(x, s, b, mean, inv)
    # the 16-bit types round once, at the store: half an ulp of the result, fp32 terms beside it
    lim = ref.U[dtype] / 2 * 1.01 * y.abs() + 64 * 2.0 ** -24 * terms + ref.TINY[dtype]
    assert ((Y.double().cpu() - y).abs() <= lim).all()
    # without B
    Y0, _, _ = gs_cuda.gs_layer_norm(Xd, Sd)
    y0 = ref.layer_norm(x, s, None, 1e-5)[0]
    lim = ref.U[dtype] / 2 * 1.01 * y0.abs() + 64 * 2.0 ** -24 * terms + ref.TINY[dtype]
    assert ((Y0.double().cpu() - y0).abs() <= lim).all()
    # gradient, from the statistics the kernel itself gave
    m64, i64 = M.double().cpu(), I.double().cpu()
    grads, sums = ref.layer_norm_backward(dy, x, s, m64, i64)
    got = gs_cuda.gs_layer_norm_backward(dYd, Xd, Sd, M, I)
    level = (x.abs() + m64.abs()) * i64      # xhat's terms before they cancel
    extra = [i64 * level * (dy * s).abs().mean(1, keepdim=True) * 2,
             (dy.abs() * level).sum(0), 0.0]
    for name, a, r, t, e in zip(("dX", "dScale", "dB"), got, grads, sums, extra):
        ref.check(a, r, t + e, dtype, name)
    # the same bits again
    for a, c in zip(got, gs_cuda.gs_layer_norm_backward(dYd, Xd, Sd, M, I)):
        assert torch.equal(a, c)
    assert torch.equal(Y, gs_cuda.gs_layer_norm(Xd, Sd, Bd)[0])
    assert gs_cuda.gs_device_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_layer_norm_many_rows_reduce_to_one_weight_gradient(gs_cuda, dtype):
    # more rows than row blocks, a ragged last one
    rows, D = 41003, 40
    X, S, B, dY = _norm_inputs(5, rows, D, dtype)
    Xd, Sd, dYd = X.cuda(), S.cuda(), dY.cuda()
    _, M, I = gs_cuda.gs_layer_norm(Xd, Sd)
    grads, sums = ref.layer_norm_backward(dY.double(), X.double(), S.double(), M.double().cpu(),
                                          I.double().cpu())
    for name, a, r, t in zip(("dX", "dScale", "dB"),
                             gs_cuda.gs_layer_norm_backward(dYd, Xd, Sd, M, I), grads, sums):
        ref.check(a, r, 2 * t, dtype, name)


@pytest.mark.parametrize("shift", [1, 3])
@pytest.mark.parametrize("dtype", DTYPES)
def test_layer_norm_at_odd_addresses_and_axes(gs_cuda, shift, dtype):
    # tensors that start at an element boundary only, and two normalised axes
    g = wl.rng(31)
    hold = [wl.as_dtype(g.normal(size=shift + 6 * 4 * 20), dtype).cuda() for _ in range(2)]
    X, dY = (h[shift:].view(6, 4, 20) for h in hold)
    S = wl.as_dtype(g.normal(size=shift + 80), dtype).cuda()[shift:].view(4, 20)
    Y, M, I = gs_cuda.gs_layer_norm(X, S, S, axis=1)
    Y2, M2, I2 = gs_cuda.gs_layer_norm(X.clone().view(6, 80), S.clone().view(80), S.clone().view(80))
    assert M.shape == (6, 1, 1)
    x = X.double().cpu().view(6, 80)
    s = S.double().cpu().view(80)
    y = ref.layer_norm(x, s, s, 1e-5)
    size = x.abs().mean(1, keepdim=True)
    for m, i in ((M.view(6, 1), I.view(6, 1)), (M2, I2)):
        ref.check(m, y[1], size, "float32", "mean")
        ref.check(i, y[2], y[2] * (1 + size * y[2]), "float32", "inv")
    ref.check(Y.view(6, 80), y[0], _norm_terms(x, s, s, y[1], y[2]), dtype, "Y")
    a = gs_cuda.gs_layer_norm_backward(dY, X, S, M, I, axis=1)
    b = gs_cuda.gs_layer_norm_backward(dY.clone(), X.clone(), S.clone(), M, I, axis=1)
    for u, v in zip(a, b):
        scale = v.abs().amax().double().item()
        assert (u.double() - v.double()).abs().amax().item() <= 2 * ref.U[dtype] * scale


def test_layer_norm_gradient_against_differences(gs_cuda):
    g = wl.rng(77)
    X, S, B, W = _norm_inputs(78, 6, 96, "float32")
    x, s, b, w = (t.double() for t in (X, S, B, W))
    Y, M, I = gs_cuda.gs_layer_norm(X.cuda(), S.cuda(), B.cuda())
    dX, dS, dB = (t.double().cpu() for t in gs_cuda.gs_layer_norm_backward(
        W.cuda(), X.cuda(), S.cuda(), M, I))
    f = lambda x_, s_, b_: (ref.layer_norm(x_, s_, b_, 1e-5)[0] * w).sum()
    h = 1e-5
    for _ in range(4):
        vx, vs, vb = (torch.from_numpy(g.normal(size=t.shape)) for t in (x, s, b))
        num = (f(x + h * vx, s + h * vs, b + h * vb) - f(x - h * vx, s - h * vs, b - h * vb)) / (2 * h)
        ana = (dX * vx).sum() + (dS * vs).sum() + (dB * vb).sum()
        size = (dX * vx).abs().sum() + (dS * vs).abs().sum() + (dB * vb).abs().sum()
        # central differences are off by h^2 f'''/6 ~ 1e-9, the kernel by fp32 ulps
        assert abs(num - ana) <= 1e-5 * size


def test_layer_norm_constant_rows_infinities_and_nan(gs_cuda):
    X = torch.full((4, 100), 3.25, device="cuda")
    X[1, 5] = float("inf")
    X[2, 7] = float("nan")
    S = torch.ones(100, device="cuda")
    B = torch.full((100,), 0.5, device="cuda")
    Y, M, I = gs_cuda.gs_layer_norm(X, S, B)
    assert torch.equal(Y[0], B) and torch.equal(Y[3], B)       # nothing but B is left
    assert abs(I[0].item() - 1e-5 ** -0.5) < 1e-3
    assert torch.isnan(Y[1]).all() and torch.isnan(Y[2]).all()  # other rows are untouched


@pytest.mark.parametrize("dtype,D", [("float32", 37), ("float32", 132), ("bfloat16", 264),
                                     ("bfloat16", 2100)])
def test_layer_norm_gradient_of_constant_rows_whose_level_overflows(gs_cuda, dtype, D):
    # mean * inv is beyond fp32, x - mean is zero: only lanes behind a row's end see it
    level, inv = 2.0 ** 112, 2.0 ** 20
    g = wl.rng(31)
    dY = wl.as_dtype(g.normal(size=(3, D)), dtype)
    scale = wl.as_dtype(g.normal(size=D), dtype)
    X = torch.full((3, D), level, dtype=dY.dtype)
    stat = lambda v: torch.full((3, 1), v).cuda()
    dX, dScale, dB = gs_cuda.gs_layer_norm_backward(dY.cuda(), X.cuda(), scale.cuda(), stat(level),
                                                    stat(inv))
    gw = dY.double() * scale.double()
    want = inv * (gw - gw.mean(1, keepdim=True))
    # a rounding of the output and fp32 roundings of a sum of D terms
    unit = 2.0 ** -23 if dtype == "float32" else 2.0 ** -8
    bound = unit * want.abs() + 2.0 ** -23 * inv * (gw.abs() + gw.abs().sum(1, keepdim=True))
    assert ((dX.cpu().double() - want).abs() <= bound).all()
    assert (dScale == 0).all() and torch.isfinite(dB.float()).all()


def test_layer_norm_large_level_keeps_its_variance(gs_cuda):
    # mean 4096 with deviations of 1: a one-pass sum of squares would lose the variance
    g = wl.rng(3)
    x = 4096.0 + g.normal(size=(8, 512))
    X = wl.as_dtype(x, "float32")
    _, M, I = gs_cuda.gs_layer_norm(X.cuda(), torch.ones(512, device="cuda"))
    inv = ref.layer_norm(X.double(), torch.ones(512).double(), None, 1e-5)[2]
    # the mean is off by at most 2^-24 * 4096 * 16, which adds its square to the variance
    assert ((I.double().cpu() - inv).abs() <= 1e-4 * inv).all()


def test_layer_norm_empty(gs_cuda):
    S = torch.ones(16, device="cuda")
    X = torch.empty((0, 16), device="cuda")
    Y, M, I = gs_cuda.gs_layer_norm(X, S)
    assert Y.shape == (0, 16) and M.shape == (0, 1)
    dX, dS, dB = gs_cuda.gs_layer_norm_backward(X, X, S, M, I)
    assert dX.shape == (0, 16) and not dS.any() and not dB.any()


# ------------------------------------------------------------------ dropout

def _dropout_exact(x, residual, ratio, seed, offset):
    words = np.array(ref.philox_words(x.numel(), seed, offset), dtype=np.int64)
    keep = torch.from_numpy(words >= int(np.floor(ratio * 2 ** 32 + 0.5))).view(x.shape)
    y = torch.where(keep, x.double() / (1.0 - ratio), 0.0)
    return (y if residual is None else y + residual.double()), keep


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 1000, 4099])
@pytest.mark.parametrize("with_residual", [False, True])
def test_dropout_matches_the_generator(gs_cuda, n, dtype, with_residual):
    g = wl.rng(n)
    X = wl.as_dtype(g.normal(size=n), dtype)
    R = wl.as_dtype(g.normal(size=n), dtype) if with_residual else None
    seed, offset = 0xDEADBEEF12345678, (1 << 40) + 17
    y, keep = _dropout_exact(X, R, 0.3, seed, offset)
    Y = gs_cuda.gs_dropout(X.cuda(), 0.3, seed, offset, residual=None if R is None else R.cuda())
    got = Y.double().cpu()
    # the scale, the product and the sum in fp32, one rounding to the type
    size = X.double().abs() / 0.7 + (R.double().abs() if R is not None else 0.0)
    assert ((got - y).abs() <= ref.U[dtype] / 2 * 1.01 * y.abs() + 4 * 2.0 ** -24 * size
            + ref.TINY[dtype]).all()
    if R is None:
        assert torch.equal(got != 0, keep & (X != 0))


@pytest.mark.parametrize("shift", [0, 1, 2, 5])
@pytest.mark.parametrize("dtype", DTYPES)
def test_dropout_mask_does_not_depend_on_address_or_type(gs_cuda, shift, dtype):
    n = 3001
    one = torch.ones(n + shift, dtype=DT[dtype], device="cuda")[shift:]
    base = gs_cuda.gs_dropout(torch.ones(n, device="cuda"), 0.4, 5, 9) != 0
    assert torch.equal(gs_cuda.gs_dropout(one, 0.4, 5, 9) != 0, base)
    out = torch.empty(n + shift, dtype=DT[dtype], device="cuda")[shift:]
    gs_cuda.gs_dropout(one.clone(), 0.4, 5, 9, out=out)
    assert torch.equal(out != 0, base)


def test_dropout_gradient_repeats_the_mask(gs_cuda):
    X = torch.randn(100, 77, device="cuda")
    dY = torch.randn(100, 77, device="cuda")
    Y = gs_cuda.gs_dropout(X, 0.25, 11, 3)
    dX = gs_cuda.gs_dropout(dY, 0.25, 11, 3)
    keep = Y != 0
    assert torch.equal(dX, torch.where(keep, dY * (1.0 / 0.75), 0.0))
    # against differences: Y is linear in X
    h = 0.5
    up = gs_cuda.gs_dropout(X + h * dY, 0.25, 11, 3).double()
    down = gs_cuda.gs_dropout(X - h * dY, 0.25, 11, 3).double()
    size = (X.abs() + dY.abs()).double()
    assert (((up - down) / (2 * h) - dX.double()).abs() <= 16 * 2.0 ** -24 * size).all()


def test_dropout_ratio_zero_in_place_and_non_finite_drops(gs_cuda):
    X = torch.randn(1001, device="cuda")
    assert torch.equal(gs_cuda.gs_dropout(X, 0.0, 1, 2), X)
    keep = gs_cuda.gs_dropout(torch.ones_like(X), 0.5, 1, 2) != 0
    bad = torch.where(keep, X, float("nan"))
    bad[~keep & (X > 0)] = float("inf")
    R = torch.randn(1001, device="cuda")
    want = torch.where(keep, R + X * 2.0, R)
    assert torch.equal(gs_cuda.gs_dropout(bad, 0.5, 1, 2, residual=R), want)
    inplace = bad.clone()
    assert gs_cuda.gs_dropout(inplace, 0.5, 1, 2, residual=R, out=inplace) is inplace
    assert torch.equal(inplace, want)
    into = R.clone()
    gs_cuda.gs_dropout(bad, 0.5, 1, 2, residual=into, out=into)
    assert torch.equal(into, want)


def test_dropout_share_of_kept_elements(gs_cuda):
    n = 1 << 22
    for k, ratio in enumerate((0.1, 0.5, 0.9)):
        Y = gs_cuda.gs_dropout(torch.ones(n, device="cuda"), ratio, 123 + k, 0)
        share = (Y == 0).double().mean().item()
        assert abs(share - ratio) <= 6 * (ratio * (1 - ratio) / n) ** 0.5   # six deviations
    a = gs_cuda.gs_dropout(torch.ones(n, device="cuda"), 0.5, 1, 0) != 0
    for seed, offset in ((2, 0), (1, 1), (1, 1 << 33), (1 + (1 << 32), 0)):
        b = gs_cuda.gs_dropout(torch.ones(n, device="cuda"), 0.5, seed, offset) != 0
        assert abs((a == b).double().mean().item() - 0.5) <= 6 * (0.25 / n) ** 0.5


def test_calls_run_on_the_current_stream(gs_cuda):
    side = torch.cuda.Stream()
    X = torch.randn(4096, 256, device="cuda")
    S = torch.ones(256, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Y, M, I = gs_cuda.gs_layer_norm(X, S)
        Z = gs_cuda.gs_dropout(Y, 0.5, 1, 1, residual=X)
    torch.cuda.current_stream().wait_stream(side)
    Y2, _, _ = gs_cuda.gs_layer_norm(X, S)
    assert torch.equal(Y, Y2) and torch.equal(Z, gs_cuda.gs_dropout(Y2, 0.5, 1, 1, residual=X))
