"""64-bit references of the feed-forward operators and the error bounds the tests hold the
kernels to.

Bounds.  With h the half step of the type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32) and A the sum of the
absolute values of a result's terms, a result rounded once is off by at most

    h |ref| (1 + 2^-6) + C 2^-24 A + the type's smallest half step

and one whose factors are rounded to the type as well by h A more.  C covers fp32 sums of n terms:
8 sqrt(n) for roundings to nearest (eight deviations of n independent half steps), n / 8 for
tensor cores that add sixteen products at a time and cut the sum off (up to two half steps for
each of n / 16), and 64 for the activation (two approximations of 2 ulps each behind an argument
that is off by a few) and the formulas around it.
"""
import math

import torch

HALF = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 1e-37, "float16": 2.0 ** -25, "bfloat16": 1e-37}
OVER = {"float32": 2.0 ** 128 - 2.0 ** 103, "float16": 65520.0, "bfloat16": 2.0 ** 128 - 2.0 ** 119}
DT = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


def terms(n):
    return 8 * math.sqrt(n) + n / 8 + 64


def check(got, ref, A, dtype, C, rounded=0.0, what=""):
    """``rounded``: the absolute sum of terms whose factors are rounded to the type, once each."""
    got = got.detach().to(torch.float64).cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    fine = ~(torch.isnan(ref) | inf)
    limit = HALF[dtype] * (ref.abs() * (1 + 2.0 ** -6) + rounded) + C * 2.0 ** -24 * A + TINY[dtype]
    err = (got - ref).abs()
    # half a step above the type's largest value and beyond, rounding to nearest gives infinity
    over = (ref.abs() + limit >= OVER[dtype]) & torch.isinf(got) & (got.sign() == ref.sign())
    bad = fine & ~(err <= limit) & ~over
    if bad.any():
        i = int(torch.argmax(torch.where(bad, err / limit, torch.zeros_like(err))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at flat {i}: "
                             f"got {got.flatten()[i]!r}, ref {ref.flatten()[i]!r}, "
                             f"bound {limit.flatten()[i]!r}")


def wide(t):
    return None if t is None else t.detach().cpu().to(torch.float64)


# ------------------------------------------------------------------ gated projections

def act(name, g):
    """act(g) and its slope in 64 bits."""
    if name == "silu":
        r = torch.sigmoid(g)
        return g * r, r + g * r * (1 - r)
    if name == "gelu":
        phi = torch.special.ndtr(g)
        return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g ** 3))
        return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 2 * k * (1 + 0.134145 * g * g)
    if name == "relu":
        return torch.where(g < 0, torch.zeros_like(g), g), (g > 0).to(g.dtype)
    if name == "sigmoid":
        r = torch.sigmoid(g)
        return r, r * (1 - r)
    return g, torch.ones_like(g)


def gated(X, Wg, Wu, bg, bu, name):
    """(H, G, U) and the absolute sums of each."""
    x, wg, wu = (wide(t) for t in (X, Wg, Wu))
    G, U = x @ wg.T, x @ wu.T
    aG, aU = x.abs() @ wg.abs().T, x.abs() @ wu.abs().T
    if bg is not None:
        G, U, aG, aU = G + wide(bg), U + wide(bu), aG + wide(bg).abs(), aU + wide(bu).abs()
    a, _ = act(name, G)
    # no activation's slope is above 1.13
    return (a * U, G, U), (1.13 * aG * U.abs() + a.abs() * aU + (aG + 1) * U.abs() * 0.25, aG, aU)


def check_gated(got, X, Wg, Wu, bg, bu, name, dtype, what=""):
    refs, sums = gated(X, Wg, Wu, bg, bu, name)
    C = terms(X.shape[-1])
    for t, r, A, part in zip(got, refs, sums, "HGU"):
        check(t, r, A, dtype, C, what=f"{what} {part}")


def gated_backward(dH, X, Wg, Wu, G, U, name):
    """[dX, dWg, dWu, dbg, dbu], the absolute sums of the terms as they are, and of the terms with
    a slope of 1 at least, which the slope's own error is small beside."""
    dh, x, wg, wu, g, u = (wide(t) for t in (dH, X, Wg, Wu, G, U))
    a, da = act(name, g)
    dG, dU = dh * u * da, dh * a
    refs = [dG @ wg + dU @ wu, dG.T @ x, dU.T @ x, dG.sum(0), dU.sum(0)]

    def sums(p, q):
        return [p @ wg.abs() + q @ wu.abs(), p.T @ x.abs(), q.T @ x.abs(), p.sum(0), q.sum(0)]

    plain = sums(dG.abs(), dU.abs())
    floor = sums((dh * u).abs() * (da.abs() + 1), dh.abs() * (a.abs() + 0.25))
    return refs, plain, floor


def check_gated_backward(got, dH, X, Wg, Wu, G, U, name, dtype, what=""):
    refs, plain, floor = gated_backward(dH, X, Wg, Wu, G, U, name)
    rows, F = G.numel() // max(G.shape[-1], 1), G.shape[-1]
    counts = [2 * F, rows, rows, rows, rows]
    for i, t in enumerate(got):
        # dG and dU are factors of the products in the type; the biases' sums take them unrounded
        rounded = plain[i] * (1 + 2.0 ** -6) if i < 3 and dtype != "float32" else 0.0
        check(t, refs[i], floor[i], dtype, terms(counts[i]), rounded,
              f"{what} {['dX', 'dWg', 'dWu', 'dbg', 'dbu'][i]}")


# ------------------------------------------------------------------ norms around a branch

def _normed(v, A, kind, eps):
    """v's rows normalised, mean, reciprocal deviation, and the absolute sums of the first: an
    error of A per element moves the mean by its mean and the deviation by its rms."""
    D = v.shape[1]
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    c = v - mean
    inv = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    rms = (A * A).mean(1, keepdim=True).sqrt()
    return c * inv, mean, inv, inv * (A + rms * (1 + (c * inv).abs()))


def by_row(gate, rows, D):
    if gate is None:
        return torch.ones((1, D), dtype=torch.float64)
    g = wide(gate).reshape(-1, D)
    return g.repeat_interleave(rows // g.shape[0], 0)


def residual_norm(X, Z, Scale, B, gate, z_scale, z_B, kind, alpha, eps):
    """(S, Y, Stats) and their absolute sums."""
    x, z = wide(X), wide(Z)
    rows, D = x.shape
    zero, one = torch.zeros((rows, 1), dtype=torch.float64), torch.ones((rows, 1), dtype=torch.float64)
    stats, A = [zero, one], z.abs()
    if z_scale is not None:
        z, m, i, A = _normed(z, A, kind, eps)
        b = wide(z_B) if z_B is not None else torch.zeros(D, dtype=torch.float64)
        z, A, stats = z * wide(z_scale) + b, A * wide(z_scale).abs() + b.abs(), [m, i]
    g = by_row(gate, rows, D)
    S, A = alpha * x + g * z, abs(alpha) * x.abs() + g.abs() * A
    y, m, i, AY = _normed(S, A, kind, eps)
    b = wide(B) if B is not None else torch.zeros(D, dtype=torch.float64)
    Y, AY = y * wide(Scale) + b, AY * wide(Scale).abs() + b.abs()
    stats += [m, i]
    rz, rs = wide(Z).abs().square().mean(1, keepdim=True).sqrt(), (A * A).mean(1, keepdim=True).sqrt()
    spread = [rz, stats[1] * (1 + stats[1] * rz), rs, i * (1 + i * rs)]
    return (S, Y, torch.cat(stats, 1)), (A, AY, torch.cat(spread, 1))


def _pull(w, aw, hat, inv, kind):
    """N(w, hat, inv) and its absolute sums."""
    level = w.mean(1, keepdim=True) if kind == "layer" else 0.0
    out = inv * (w - level - hat * (w * hat).mean(1, keepdim=True))
    A = inv * (aw + aw.mean(1, keepdim=True) + hat.abs() * (aw * hat.abs()).mean(1, keepdim=True))
    return out, A


def residual_norm_backward(dS, dY, S, Z, Stats, Scale, gate, z_scale, z_B, kind, alpha):
    """Dicts of the gradients and of their absolute sums."""
    dy, s, z, st = wide(dY), wide(S), wide(Z), wide(Stats)
    rows, D = s.shape
    hat, inv = (s - st[:, 2:3]) * st[:, 3:4], st[:, 3:4]
    # the subtractions s - mean and z - mean lose as many digits as the means are large
    ahat = (s.abs() + st[:, 2:3].abs()) * inv
    w = dy * wide(Scale)
    ds, A = _pull(w, w.abs(), hat, inv, kind)
    A = A + inv * (ahat * (w * hat).mean(1, keepdim=True).abs()
                   + hat.abs() * (w.abs() * ahat).mean(1, keepdim=True))
    if dS is not None:
        ds, A = ds + wide(dS), A + wide(dS).abs()
    out = {"dX": (alpha * ds, abs(alpha) * A),
           "dScale": ((dy * hat).sum(0), (dy.abs() * ahat).sum(0)), "dB": (dy.sum(0), dy.abs().sum(0))}
    zhat, azh = (z - st[:, 0:1]) * st[:, 1:2], (z.abs() + st[:, 0:1].abs()) * st[:, 1:2]
    zs = wide(z_scale) if z_scale is not None else torch.ones(D, dtype=torch.float64)
    zb = wide(z_B) if z_B is not None else torch.zeros(D, dtype=torch.float64)
    g = by_row(gate, rows, D)
    if gate is not None:
        n = gate.numel() // D
        per = lambda t: t.reshape(n, rows // n, D).sum(1).reshape(gate.shape)
        out["dgate"] = (per(ds * (zhat * zs + zb)), per(A * (azh * zs.abs() + zb.abs())))
    e, A = ds * g, A * g.abs()
    if z_scale is not None:
        out["dz_scale"], out["dz_B"] = ((e * zhat).sum(0), (A * azh).sum(0)), (e.sum(0), A.sum(0))
        w, aw, inv = e * zs, A * zs.abs(), st[:, 1:2]
        e, A = _pull(w, aw, zhat, inv, kind)
        A = A + inv * (azh * (w * zhat).mean(1, keepdim=True).abs()
                       + zhat.abs() * (w.abs() * azh).mean(1, keepdim=True))
    out["dZ"] = (e, A)
    return out
