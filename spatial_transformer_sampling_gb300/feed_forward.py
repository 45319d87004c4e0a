"""Binding of the feed-forward operators of libgs (include/gs.h): the gated projections of a
transformer block's feed-forward half, and the norms on both sides of a branch fused with its
gate and the scaled residual sum, each with its gradient.  As in block.py the functions only
check and marshal; every step of the computation runs in libgs's kernels.
"""
import ctypes
import functools

from . import GsError, ResidualNormAttrs, _ok, _shape_error, load_library
from .block import _check_f32, _check_input, _check_like, _host, _p, _scratch

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4, "identity": 5}
NORM_KINDS = {"layer": 0, "rms": 1}


def _launch(name, device, *args):
    """Calls an entry point on the current stream of ``device``, whichever device is current."""
    h = _host()
    f, index = getattr(h.lib, name), device.index
    if h.torch._C._cuda_getDevice() == index:
        status = f(*args, h.stream(index))
    else:
        with h.torch.cuda.device(device):
            status = f(*args, h.stream(index))
    if status:
        raise GsError(status, name)


def _choice(table, value, what):
    if value not in table:
        raise ValueError(f"{what} must be one of {', '.join(table)}, not {value!r}")
    return table[value]


# ------------------------------------------------------------------ gated projections

@functools.lru_cache(maxsize=256)
def _gated_bytes(rows, D, F, code, backward):
    n = ctypes.c_size_t(0)
    name = ("gs_gated_linear_backward_workspace_size" if backward
            else "gs_gated_linear_workspace_size")
    _ok(getattr(load_library(), name)(rows, D, F, code, ctypes.byref(n)), name)
    return int(n.value)


def _dtype_code(dtype):
    codes = _host().codes
    if dtype not in codes:
        raise TypeError(f"unsupported dtype {dtype}")
    return codes[dtype]


def gs_gated_linear_workspace_size(rows, D, F, dtype):
    """Workspace bytes gs_gated_linear needs."""
    return _gated_bytes(rows, D, F, _dtype_code(dtype), False)


def gs_gated_linear_backward_workspace_size(rows, D, F, dtype):
    """Workspace bytes gs_gated_linear_backward needs."""
    return _gated_bytes(rows, D, F, _dtype_code(dtype), True)


def _check_weights(X, Wg, Wu):
    """(rows, D, F) of X (..., D) and Wg, Wu (F, D)."""
    _check_input(X)
    if X.dim() < 1 or X.shape[-1] == 0:
        raise ValueError(f"X must be (..., D) with D > 0, got {tuple(X.shape)}")
    D = X.shape[-1]
    if Wg.dim() != 2 or Wg.shape[1] != D:
        raise ValueError(f"Wg must be (F, D={D}), got {tuple(Wg.shape)}")
    F = Wg.shape[0]
    _check_like(X, "Wg", Wg, (F, D))
    _check_like(X, "Wu", Wu, (F, D))
    return X.numel() // D, D, F


class _GatedPlan:
    """What the shapes and the dtype alone decide.  Kept per signature, as attention's plans are:
    working it out takes longer than a launch."""

    def __init__(self, X, Wg, Wu):
        self.rows, self.D, self.F = _check_weights(X, Wg, Wu)
        self.code = _host().codes[X.dtype]
        self.weights = (self.F, self.D)
        self.outputs = X.shape[:-1] + (self.F,)
        self.bytes = [_gated_bytes(self.rows, self.D, self.F, self.code, b) for b in (False, True)]


_GATED_PLANS = {}
_MOST_PLANS = 256


def _fits(t, dtype, device, shape):
    """A contiguous tensor of this dtype, device and shape (_check_like says what does not fit)."""
    return t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous()


def _gated_plan(X, Wg, Wu):
    key = (X.shape, Wg.shape, X.dtype)
    plan = _GATED_PLANS.get(key)
    if plan is None:
        plan = _GatedPlan(X, Wg, Wu)
        if len(_GATED_PLANS) >= _MOST_PLANS:
            _GATED_PLANS.clear()
        _GATED_PLANS[key] = plan
    dtype, device = X.dtype, X.device
    if not (device.type == "cuda" and X.is_contiguous() and _fits(Wg, dtype, device, plan.weights)
            and _fits(Wu, dtype, device, plan.weights)):
        _check_weights(X, Wg, Wu)
    return plan, dtype, device


def gs_gated_linear(X, Wg, Wu, bg=None, bu=None, activation="silu", keep=False, out=None,
                    workspace="auto"):
    """H = act(X Wg^T + bg) * (X Wu^T + bu), the gated projections of a feed-forward block.

    X (..., D), Wg and Wu (F, D), bg and bu (F) or both None; ``activation`` is "silu", "gelu",
    "gelu_tanh", "relu", "sigmoid" or "identity".  H is (..., F); with ``keep`` the call returns
    (H, G, U), where G and U are the two projections, which the backward pass takes.
    ``out``: a tensor for H that overlaps no input.
    ``workspace``: "auto", or a device tensor of at least gs_gated_linear_workspace_size bytes."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        _choice(ACTIVATIONS, activation, "activation")
    plan, dtype, device = _gated_plan(X, Wg, Wu)
    if bg is not None or bu is not None:
        if bg is None or bu is None:
            raise ValueError("bg and bu go together")
        _check_like(X, "bg", bg, (plan.F,))
        _check_like(X, "bu", bu, (plan.F,))
    shape = plan.outputs
    if out is None:
        out = X.new_empty(shape)
    elif not _fits(out, dtype, device, shape):
        _check_like(X, "out", out, shape)
    G = U = None
    if keep:
        G, U = X.new_empty(shape), X.new_empty(shape)
    ws, have, _keep = _scratch(workspace, plan.bytes[0], X)
    _launch("gs_gated_linear", device, X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), _p(bg), _p(bu),
            plan.rows, plan.D, plan.F, act, plan.code, ws, have, out.data_ptr(), _p(G), _p(U))
    return (out, G, U) if keep else out


def gs_gated_linear_backward(dH, X, Wg, Wu, G, U, activation="silu", bias=False, workspace="auto"):
    """Gradient of gs_gated_linear from the G and U that it kept: [dX, dWg, dWu], and with
    ``bias`` dbg and dbu after them."""
    act = _choice(ACTIVATIONS, activation, "activation")
    plan, dtype, device = _gated_plan(X, Wg, Wu)
    for t, what in ((dH, "dH"), (G, "G"), (U, "U")):
        if not _fits(t, dtype, device, plan.outputs):
            _check_like(X, what, t, plan.outputs)
    made = [X.new_empty(X.shape), X.new_empty(plan.weights), X.new_empty(plan.weights)]
    if bias:
        made += [X.new_empty((plan.F,)), X.new_empty((plan.F,))]
    ws, have, _keep = _scratch(workspace, plan.bytes[1], X)
    out = [t.data_ptr() for t in made] + ([] if bias else [None, None])
    _launch("gs_gated_linear_backward", device, dH.data_ptr(), X.data_ptr(), Wg.data_ptr(),
            Wu.data_ptr(), G.data_ptr(), U.data_ptr(), plan.rows, plan.D, plan.F, act, plan.code, ws,
            have, *out)
    return made


# ------------------------------------------------------------------ norms around a branch

def _check_norm(X, Z, Scale, gate, z_scale, z_B, B=None):
    """(rows, D, groups of the gate) of tensors that fit together."""
    _check_input(X)
    if X.dim() < 1:
        raise ValueError("X must be (..., D)")
    D = X.shape[-1]
    rows = 1
    for n in X.shape[:-1]:
        rows *= n
    _check_like(X, "Z", Z, X.shape)
    _check_like(X, "Scale", Scale, (D,))
    groups = 0
    if gate is not None:
        if gate.dim() not in (1, 2) or gate.shape[-1] != D:
            raise ValueError(f"gate must be (D={D}) or (groups, D), got {tuple(gate.shape)}")
        groups = gate.shape[0] if gate.dim() == 2 else 1
        if groups == 0 or rows % groups:
            raise ValueError(f"{groups} rows of a gate do not divide {rows} rows")
        _check_like(X, "gate", gate, gate.shape)
    if z_scale is not None:
        _check_like(X, "z_scale", z_scale, (D,))
    if z_B is not None:
        if z_scale is None:
            raise ValueError("z_B needs z_scale")
        _check_like(X, "z_B", z_B, (D,))
    if B is not None:
        _check_like(X, "B", B, (D,))
    return rows, D, groups


class _NormPlan:
    """What the shapes, the dtype and the numbers alone decide."""

    def __init__(self, X, Z, Scale, gate, z_scale, z_B, kind, alpha, epsilon):
        rows, D, groups = _check_norm(X, Z, Scale, gate, z_scale, z_B)
        self.attrs = ResidualNormAttrs(rows, D, groups, _choice(NORM_KINDS, kind, "kind"), alpha,
                                       epsilon)
        self.ref = ctypes.byref(self.attrs)
        self.code = _host().codes[X.dtype]
        self.width = (D,)
        self.stats = X.shape[:-1] + (4,)
        self.bytes = None

    def workspace(self):
        if self.bytes is None:
            at = self.attrs
            self.bytes = _residual_norm_bytes(at.rows, at.D, at.groups, self.code)
        return self.bytes


_NORM_PLANS = {}


def _norm_plan(X, Z, Scale, B, gate, z_scale, z_B, kind, alpha, epsilon):
    alpha, epsilon = float(alpha), float(epsilon)   # a plan holds numbers
    key = (X.shape, X.dtype, None if gate is None else gate.shape, kind, alpha, epsilon)
    plan = _NORM_PLANS.get(key)
    if plan is None:
        plan = _NormPlan(X, Z, Scale, gate, z_scale, z_B, kind, alpha, epsilon)
        if len(_NORM_PLANS) >= _MOST_PLANS:
            _NORM_PLANS.clear()
        _NORM_PLANS[key] = plan
    dtype, device, width = X.dtype, X.device, plan.width
    if not (device.type == "cuda" and X.is_contiguous() and _fits(Z, dtype, device, X.shape)
            and _fits(Scale, dtype, device, width)
            and (B is None or _fits(B, dtype, device, width))
            and (gate is None or _fits(gate, dtype, device, gate.shape))
            and (z_scale is None or _fits(z_scale, dtype, device, width))
            and (z_B is None or z_scale is not None and _fits(z_B, dtype, device, width))):
        _check_norm(X, Z, Scale, gate, z_scale, z_B, B)
    return plan, dtype, device


def gs_residual_norm(X, Z, Scale, B=None, gate=None, z_scale=None, z_B=None, kind="layer",
                     alpha=1.0, epsilon=1e-5):
    """S = alpha X + gate * z', Y = norm(S) * Scale + B with z' = norm(Z) * z_scale + z_B, or Z
    without z_scale: the norm after a branch Z, its gate, the scaled residual sum and the norm
    before the next branch, in one pass.  Returns (S, Y, Stats).

    X and Z (..., D); Scale, B, z_scale and z_B (D); ``gate`` (D), or (groups, D) where
    rows / groups consecutive rows share one; ``kind`` "layer" or "rms", of both norms.  Stats
    (..., 4) float32 holds the mean and reciprocal deviation of Z (0 and 1 without z_scale) and
    those of S, which the backward pass takes (where D is 0, NaN)."""
    plan, dtype, device = _norm_plan(X, Z, Scale, B, gate, z_scale, z_B, kind, alpha, epsilon)
    torch = _host().torch
    S, Y = torch.empty_like(X), torch.empty_like(X)
    stats = torch.empty(plan.stats, dtype=torch.float32, device=device)
    _launch("gs_residual_norm", device, X.data_ptr(), Z.data_ptr(), _p(gate), _p(z_scale), _p(z_B),
            Scale.data_ptr(), _p(B), plan.ref, plan.code, S.data_ptr(), Y.data_ptr(),
            stats.data_ptr())
    if plan.attrs.D == 0:   # the call writes nothing; the mean of no element
        stats.fill_(float("nan"))
    return S, Y, stats


@functools.lru_cache(maxsize=256)
def _residual_norm_bytes(rows, D, groups, code):
    n = ctypes.c_size_t(0)
    at = ResidualNormAttrs(rows, D, groups, 0, 1.0, 0.0)
    name = "gs_residual_norm_backward_workspace_size"
    _ok(getattr(load_library(), name)(ctypes.byref(at), code, ctypes.byref(n)), name)
    return int(n.value)


def gs_residual_norm_backward_workspace_size(rows, D, groups, dtype):
    """Workspace bytes gs_residual_norm_backward needs with a gate of ``groups`` rows (0: none)."""
    return _residual_norm_bytes(rows, D, groups, _dtype_code(dtype))


def gs_residual_norm_backward(dS, dY, S, Z, Stats, Scale, bias=False, gate=None, z_scale=None,
                              z_B=None, kind="layer", alpha=1.0, workspace="auto"):
    """Gradient of gs_residual_norm: a dict of dX, dZ, dScale, dB (with ``bias``), dgate, dz_scale
    and dz_B, the last three for what was given.  ``dS`` (None: zeros) is what reaches S
    otherwise; S and Stats are the forward call's.  ``workspace``: "auto", or a device tensor of at
    least gs_residual_norm_backward_workspace_size bytes."""
    plan, dtype, device = _norm_plan(S, Z, Scale, None, gate, z_scale, z_B, kind, alpha, 0.0)
    if dS is not None and not _fits(dS, dtype, device, S.shape):
        _check_like(S, "dS", dS, S.shape)
    if not _fits(dY, dtype, device, S.shape):
        _check_like(S, "dY", dY, S.shape)
    _check_f32(Stats, plan.stats, "Stats", S)
    like, width = _host().torch.empty_like, plan.width
    made = {"dX": like(S), "dZ": like(S), "dScale": S.new_empty(width)}
    if bias:
        made["dB"] = S.new_empty(width)
    if gate is not None:
        made["dgate"] = like(gate)
    if z_scale is not None:
        made["dz_scale"] = S.new_empty(width)
    if z_B is not None:
        made["dz_B"] = S.new_empty(width)
    ws, have, _keep = _scratch(workspace, plan.workspace(), S)
    out = [_p(made.get(k)) for k in ("dX", "dZ", "dgate", "dz_scale", "dz_B", "dScale", "dB")]
    _launch("gs_residual_norm_backward", device, _p(dS), dY.data_ptr(), S.data_ptr(), Z.data_ptr(),
            Stats.data_ptr(), _p(gate), _p(z_scale), _p(z_B), Scale.data_ptr(), plan.ref, plan.code,
            ws, have, *out)
    return made
