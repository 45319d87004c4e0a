"""The feed-forward half of a transformer block on real shapes: cases, inputs, plain forms and
exact values.

Two operators, each with its directions:

  gated_linear    H = act(X Wg^T + bg) * (X Wu^T + bu), the gated projections of a feed-forward
                  block; forward (H, or H, G, U for training) and backward (dX, dWg, dWu and the
                  biases' gradients).
  residual_norm   S = alpha X + gate * norm(Z), Y = norm(S): the norm after a branch, its gate, the
                  scaled residual sum and the norm before the next branch; forward (S, Y, Stats)
                  and backward (dX, dZ, dScale, and what else was given).

With ``own`` false, ``run`` computes the plain form in elementary torch operations and 32 bits,
rounded once at the end; with ``own`` true it makes the calls of the package.
"""
import math

import torch

own = False

DT = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
EPS = 1e-5
ACTIVATIONS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid", "identity"]


# ------------------------------------------------------------------ cases

def _glu(name, direction, dtype, rows, D, F, activation, bias=False, keep=False):
    return {"name": name, "op": "gated_linear", "dir": direction, "dtype": dtype, "rows": rows,
            "D": D, "F": F, "activation": activation, "bias": bias, "keep": keep}


def _norm(name, direction, dtype, rows, D, kind, post, groups, alpha):
    """``groups``: rows of the gate, 0 for none."""
    return {"name": name, "op": "residual_norm", "dir": direction, "dtype": dtype, "rows": rows,
            "D": D, "kind": kind, "post": post, "groups": groups, "alpha": alpha}


def listed():
    return [
        # one new token: the weights are read for a single row
        _glu("glu_token", "forward", "bfloat16", 1, 1024, 4096, "silu"),
        # the pooled tokens of a few images
        _glu("glu_few_rows", "forward", "float16", 7, 384, 1536, "gelu", bias=True),
        # every pixel of a 4 x 64 x 256 x 256 feature map as a token of 64 channels, in training
        _glu("glu_pixels", "forward", "bfloat16", 4 * 256 * 256, 64, 256, "gelu_tanh", bias=True,
             keep=True),
        # a training step's tokens at a wide model width
        _glu("glu_wide", "forward", "bfloat16", 16384, 1024, 4096, "silu", keep=True),
        # a 24 x 24 grid and its summary token in 32 bits, widths that no tile divides
        _glu("glu_odd", "forward", "float32", 577, 771, 1031, "gelu", bias=True),
        # the gradient of the wide training step
        _glu("glu_bwd_wide", "backward", "bfloat16", 16384, 1024, 4096, "silu", keep=True),
        # odd rows and widths: no row is a multiple of 16 bytes
        _glu("glu_bwd_odd", "backward", "float16", 5003, 771, 1285, "gelu", bias=True, keep=True),
        # training in 32 bits
        _glu("glu_bwd_f32", "backward", "float32", 4096, 512, 2048, "silu", keep=True),
        # the pooled tokens of a few images: latency only
        _norm("norm_few_rows", "forward", "bfloat16", 7, 384, "layer", True, 1, 1.0),
        # every pixel of a 16 x 64 x 256 x 256 map, a learned scale per channel on the branch
        _norm("norm_pixels", "forward", "float32", 16 * 256 * 256, 64, "rms", False, 1, 1.0),
        # a training step's tokens, norms on both sides, a gate per item of the batch
        _norm("norm_bwd_wide", "backward", "bfloat16", 16384, 1024, "layer", True, 16, 1.0),
        # odd rows and width, a scaled residual
        _norm("norm_bwd_odd", "backward", "float32", 5003, 771, "rms", True, 0, 1.5),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_linear", "gated_linear", "residual_norm"])
    dtype = rng.choice(list(DT))
    direction = rng.choice(["forward", "backward"])
    if op == "gated_linear":
        D, F = _logint(rng, 16, 2048), _logint(rng, 16, 8192)
        if rng.random() < 0.6:                  # widths of real models are multiples of 8
            D, F = (D + 7) // 8 * 8, (F + 7) // 8 * 8
        kind = rng.choice(["serve", "few", "train", "train"])
        # as much as the largest listed forward or backward pass, in elements and in products
        most = min((16384 * 1024 * 4096) // (D * F), (1 << 26) // max(D, F))
        most = max(1, min(4 * 256 * 256, most))
        rows = {"serve": 1, "few": rng.randint(2, 64)}.get(kind) or _logint(rng, 65, max(65, most))
        rows = min(rows, most)
        if kind in ("serve", "few"):
            direction = "forward"
        return {"op": op, "dir": direction, "dtype": dtype, "rows": rows, "D": D, "F": F,
                "activation": rng.choice(ACTIVATIONS), "bias": rng.random() < 0.5,
                "keep": direction == "backward" or kind == "train"}
    D = _logint(rng, 16, 8192)
    rows = _logint(rng, 1, min(16 * 256 * 256, (1 << 24) // D))
    groups = rng.choice([0, 1, rng.randint(2, 32)])
    if groups > 1:
        rows = max(1, rows // groups) * groups
    return {"op": op, "dir": direction, "dtype": dtype, "rows": rows, "D": D,
            "kind": rng.choice(["layer", "rms"]), "post": rng.random() < 0.5, "groups": groups,
            "alpha": rng.choice([1.0, round(rng.uniform(0.5, 3.0), 3)])}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dt)

    s = {"case": dict(case)}
    rows, D = case["rows"], case["D"]
    back = case["dir"] == "backward"
    if case["op"] == "gated_linear":
        F = case["F"]
        s.update(X=normal(rows, D), Wg=normal(F, D, std=D ** -0.5), Wu=normal(F, D, std=D ** -0.5),
                 bg=None, bu=None)
        if case["bias"]:
            s.update(bg=normal(F, std=0.3), bu=normal(F, std=0.3))
        if back:
            s["dH"] = normal(rows, F)
            _, s["G"], s["U"] = _gated_linear_plain(s)
        return s
    level = torch.randn((rows, 1), generator=g, device="cuda") * 0.5
    s.update(X=(torch.randn((rows, D), generator=g, device="cuda") * 1.5 + level).to(dt),
             Z=normal(rows, D, std=0.8, mean=0.1), Scale=normal(D, std=0.2, mean=1.0),
             B=normal(D, std=0.2), gate=None, z_scale=None, z_B=None)
    if case["kind"] == "rms":
        s["B"] = None
    if case["groups"]:
        s["gate"] = normal(case["groups"], D, std=0.3, mean=0.5)
    if case["post"]:
        s["z_scale"] = normal(D, std=0.2, mean=1.0)
        s["z_B"] = normal(D, std=0.2) if case["kind"] == "layer" else None
    if back:
        s["S"], _, s["Stats"] = _residual_norm_plain(s)
        s.update(dS=normal(rows, D), dY=normal(rows, D))
    return s


# ------------------------------------------------------------------ plain forms

def _act(name, g):
    """act(g) and its derivative, in g's type."""
    if name == "silu":
        r = torch.sigmoid(g)
        return g * r, r * (1 + g * (1 - r))
    if name == "gelu":
        phi = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), (0.5 * (1 + t)
                                   + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g))
    if name == "relu":
        return torch.clamp(g, min=0), (g > 0).to(g.dtype)
    if name == "sigmoid":
        r = torch.sigmoid(g)
        return r, r * (1 - r)
    return g, torch.ones_like(g)


def _gated_linear_plain(s):
    dt, X = s["X"].dtype, s["X"].float()
    G, U = torch.matmul(X, s["Wg"].float().t()), torch.matmul(X, s["Wu"].float().t())
    if s["bg"] is not None:
        G, U = G + s["bg"].float(), U + s["bu"].float()
    H = _act(s["case"]["activation"], G)[0] * U
    return (H.to(dt), G.to(dt), U.to(dt)) if s["case"]["keep"] else H.to(dt)


def _gated_linear_backward_plain(s):
    dt, X, dH, U = s["X"].dtype, s["X"].float(), s["dH"].float(), s["U"].float()
    a, da = _act(s["case"]["activation"], s["G"].float())
    dG, dU = dH * U * da, dH * a
    out = [torch.matmul(dG, s["Wg"].float()) + torch.matmul(dU, s["Wu"].float()),
           torch.matmul(dG.t(), X), torch.matmul(dU.t(), X)]
    if s["bg"] is not None:
        out += [dG.sum(0), dU.sum(0)]
    return [t.to(dt) for t in out]


def _normed(x, kind):
    """x's rows normalised, their mean and the reciprocal of their deviation."""
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    d = x - mean
    inv = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    return d * inv, mean, inv


def _by_row(gate, rows):
    """The gate of every row: a view, or a copy of its rows where several items have their own."""
    return gate.float().repeat_interleave(rows // gate.shape[0], 0) if gate.shape[0] > 1 \
        else gate.float()


def _residual_norm_plain(s):
    dt, kind = s["X"].dtype, s["case"]["kind"]
    z = s["Z"].float()
    mean_z, inv_z = torch.zeros_like(z[:, :1]), torch.ones_like(z[:, :1])
    if s["z_scale"] is not None:
        z, mean_z, inv_z = _normed(z, kind)
        z = z * s["z_scale"].float()
        if s["z_B"] is not None:
            z = z + s["z_B"].float()
    if s["gate"] is not None:
        z = z * _by_row(s["gate"], z.shape[0])
    S = s["case"]["alpha"] * s["X"].float() + z
    y, mean_s, inv_s = _normed(S, kind)
    y = y * s["Scale"].float()
    if s["B"] is not None:
        y = y + s["B"].float()
    return S.to(dt), y.to(dt), torch.cat((mean_z, inv_z, mean_s, inv_s), 1)


def _norm_gradient(w, xhat, inv, kind):
    back = w - xhat * (w * xhat).mean(1, keepdim=True)
    if kind == "layer":
        back = back - w.mean(1, keepdim=True)
    return back * inv


def _residual_norm_backward_plain(s):
    dt, kind, case = s["X"].dtype, s["case"]["kind"], s["case"]
    mean_z, inv_z, mean_s, inv_s = s["Stats"].split(1, 1)
    dY = s["dY"].float()
    xhat = (s["S"].float() - mean_s) * inv_s
    ds = s["dS"].float() + _norm_gradient(dY * s["Scale"].float(), xhat, inv_s, kind)
    out = {"dX": case["alpha"] * ds, "dScale": (dY * xhat).sum(0)}
    if s["B"] is not None:
        out["dB"] = dY.sum(0)
    zhat = (s["Z"].float() - mean_z) * inv_z
    z = zhat
    if s["z_scale"] is not None:
        z = z * s["z_scale"].float()
        if s["z_B"] is not None:
            z = z + s["z_B"].float()
    if s["gate"] is not None:
        groups = s["gate"].shape[0]
        out["dgate"] = (ds * z).view(groups, -1, z.shape[1]).sum(1)
        ds = ds * _by_row(s["gate"], z.shape[0])
    if s["z_scale"] is not None:
        out["dz_scale"] = (ds * zhat).sum(0)
        if s["z_B"] is not None:
            out["dz_B"] = ds.sum(0)
        ds = _norm_gradient(ds * s["z_scale"].float(), zhat, inv_z, kind)
    out["dZ"] = ds
    return {k: v.to(dt) for k, v in out.items()}


# ------------------------------------------------------------------ one pass

def run(s):
    case, forward = s["case"], s["case"]["dir"] == "forward"
    if case["op"] == "gated_linear":
        if not own:
            return _gated_linear_plain(s) if forward else _gated_linear_backward_plain(s)
        import spatial_transformer_sampling_gb300 as gs
        if forward:
            return gs.gs_gated_linear(s["X"], s["Wg"], s["Wu"], s["bg"], s["bu"],
                                      activation=case["activation"], keep=case["keep"])
        return gs.gs_gated_linear_backward(s["dH"], s["X"], s["Wg"], s["Wu"], s["G"], s["U"],
                                           activation=case["activation"], bias=case["bias"])
    if not own:
        return _residual_norm_plain(s) if forward else _residual_norm_backward_plain(s)
    import spatial_transformer_sampling_gb300 as gs
    given = dict(gate=s["gate"], z_scale=s["z_scale"], z_B=s["z_B"], kind=case["kind"],
                 alpha=case["alpha"])
    if forward:
        return gs.gs_residual_norm(s["X"], s["Z"], s["Scale"], s["B"], epsilon=EPS, **given)
    return gs.gs_residual_norm_backward(s["dS"], s["dY"], s["S"], s["Z"], s["Stats"], s["Scale"],
                                        bias=s["B"] is not None, **given)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    e = 4 if case["dtype"] == "float32" else 2
    rows, D, forward = case["rows"], case["D"], case["dir"] == "forward"
    if case["op"] == "gated_linear":
        F = case["F"]
        x, h, w = rows * D, rows * F, 2 * F * D
        b = 2 * F if case["bias"] else 0
        if forward:
            return {"bytes": (x + w + b + h * (3 if case["keep"] else 1)) * e,
                    "flops": 4 * rows * D * F}
        return {"bytes": (2 * x + 3 * h + 2 * w + b) * e, "flops": 8 * rows * D * F}
    n = rows * D
    params = D * (1 + (case["kind"] == "layer")) * (2 if case["post"] else 1) + case["groups"] * D
    if forward:
        return {"bytes": (4 * n + params) * e + 16 * rows, "flops": 16 * n}
    return {"bytes": (6 * n + 2 * params) * e + 16 * rows, "flops": 30 * n}


# ------------------------------------------------------------------ 64 bits

def _exact_gated_linear(case, s):
    f64 = torch.float64
    x, wg, wu = s["X"].to(f64), s["Wg"].to(f64), s["Wu"].to(f64)
    name = case["activation"]

    def act(g):
        if name == "silu":
            return g / (1 + (-g).exp())
        if name == "gelu":
            return g * torch.special.ndtr(g)
        if name == "gelu_tanh":   # tanh(a) = 1 - 2 / (1 + e^2a)
            a = (2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)
            return g * (1 - 1 / (1 + (2 * a).exp()))
        if name == "relu":
            return torch.where(g > 0, g, torch.zeros_like(g))
        return 1 / (1 + (-g).exp()) if name == "sigmoid" else g.clone()

    if case["dir"] == "forward":
        g, u = x @ wg.T, x @ wu.T
        if case["bias"]:
            g += s["bg"].to(f64)
            u += s["bu"].to(f64)
        h = act(g) * u
        return (h, g, u) if case["keep"] else h
    g = s["G"].to(f64).requires_grad_()
    a = act(g)
    slope, = torch.autograd.grad(a.sum(), g)
    d = s["dH"].to(f64)
    to_u = a.detach() * d
    to_g = slope * d * s["U"].to(f64)
    grads = [to_g @ wg + to_u @ wu, to_g.T @ x, to_u.T @ x]
    return grads + [to_g.sum(0), to_u.sum(0)] if case["bias"] else grads


def _exact_residual_norm(case, s):
    f64 = torch.float64
    wide = {k: v.to(f64) for k, v in s.items() if torch.is_tensor(v)}
    rows, D = wide["Z"].shape
    layer = case["kind"] == "layer"
    one, zero = torch.ones((), dtype=f64, device="cuda"), torch.zeros((), dtype=f64, device="cuda")
    P, b = wide["Scale"], wide.get("B", zero)
    Pz, bz = wide.get("z_scale", one), wide.get("z_B", zero)
    groups = max(1, case["groups"])
    gate = wide.get("gate", torch.ones((1, D), dtype=f64, device="cuda"))[:, None, :]

    def grouped(t):
        return t.view(groups, rows // groups, -1)

    def statistics(t):
        m = t.sum(1, keepdim=True) / D if layer else torch.zeros((rows, 1), dtype=f64, device="cuda")
        return m, ((t ** 2).sum(1, keepdim=True) / D - m ** 2 + EPS) ** -0.5

    if case["dir"] == "forward":
        z, stats = wide["Z"], []
        if case["post"]:
            m, i = statistics(z)
            z, stats = (z - m) * i * Pz + bz, [m, i]
        else:
            stats = [torch.zeros((rows, 1), dtype=f64, device="cuda"),
                     torch.ones((rows, 1), dtype=f64, device="cuda")]
        total = wide["X"] * case["alpha"] + (grouped(z) * gate).view(rows, D)
        m, i = statistics(total)
        return total, (total - m) * i * P + b, torch.cat(stats + [m, i], 1)

    def pulled(d, t, m, i):
        """Gradient with respect to t of the sum of d * (t - m) i, m and i functions of t."""
        h = (t - m) * i
        along = (d * h).sum(1, keepdim=True)
        level = d.sum(1, keepdim=True) if layer else 0
        return i / D * (D * d - level - h * along)

    mz, iz, ms, is_ = [wide["Stats"][:, k:k + 1] for k in range(4)]
    hat_s, hat_z = (wide["S"] - ms) * is_, (wide["Z"] - mz) * iz
    ds = wide["dS"] + pulled(wide["dY"] * P, wide["S"], ms, is_)
    into = (grouped(ds) * gate).view(rows, D)
    out = {"dX": ds * case["alpha"], "dScale": torch.einsum("rd,rd->d", wide["dY"], hat_s)}
    if "B" in wide:
        out["dB"] = wide["dY"].sum(0)
    if case["groups"]:
        out["dgate"] = torch.einsum("grd,grd->gd", grouped(ds), grouped(hat_z * Pz + bz))
    if case["post"]:
        out["dz_scale"] = torch.einsum("rd,rd->d", into, hat_z)
        if "z_B" in wide:
            out["dz_B"] = into.sum(0)
    out["dZ"] = pulled(into * Pz, wide["Z"], mz, iz) if case["post"] else into
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_gated_linear if case["op"] == "gated_linear" else _exact_residual_norm)(case, s)
