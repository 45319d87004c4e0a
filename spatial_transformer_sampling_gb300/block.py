"""Binding of the transformer-block operators of libgs (include/gs.h): layer norm,
dropout with a residual sum, and attention with a learned bias by relative grid
position, each with its gradient.  As in the rest of the package the functions
only check and marshal; every step of the computation runs in libgs's kernels.
"""
import ctypes
import functools
import operator

from . import AttentionAttrs, GsError, _i64, _ok, _shape_error, _torch, load_library


class _Host:
    """torch, the library and the dtype codes, looked up once: a small call is bound by what the
    host does for it."""
    torch = lib = stream = codes = None


def _host():
    if _Host.lib is None:
        torch = _torch()
        _Host.torch = torch
        _Host.codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
        # the lookup behind torch.cuda.current_stream, without making a Stream object
        _Host.stream = torch._C._cuda_getCurrentRawStream
        _Host.lib = load_library()
    return _Host


def _p(t):
    return t.data_ptr() if t is not None else None


def _check_like(ref, what, t, shape):
    """t is contiguous, of ref's dtype and device, and of the given shape."""
    if t.dtype != ref.dtype or t.device != ref.device:
        raise ValueError("all tensors of one call share dtype and device")
    if not t.is_contiguous():
        raise ValueError("libgs takes contiguous tensors")
    if t.shape != shape:
        _shape_error(what, t.shape, shape)


def _check_input(X):
    if X.device.type != "cuda":
        raise ValueError("libgs takes CUDA tensors")
    if not X.is_contiguous():
        raise ValueError("libgs takes contiguous tensors")
    if X.dtype not in _host().codes:
        raise TypeError(f"unsupported dtype {X.dtype}")


def _scratch(workspace, nbytes, like):
    """(pointer, bytes) of a caller's workspace tensor, or with "auto" of one of `nbytes` from
    torch's allocator, and the tensor that keeps it alive."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be a tensor, None or 'auto', not {workspace!r}")
        torch = _host().torch
        workspace = (torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes
                     else None)
    elif workspace is not None and (workspace.device != like.device
                                    or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    if workspace is None:
        return None, 0, None
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _check_f32(t, shape, what, like):
    if t.dtype != _host().torch.float32 or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor on the inputs' device")
    if t.shape != shape:
        _shape_error(what, t.shape, shape)


# ------------------------------------------------------------------ layer norm

@functools.lru_cache(maxsize=256)
def _norm_dims(shape, axis):
    """(rows, D, shape of the normalised axes, shape of the statistics) of a layer norm over the
    axes of ``shape`` from ``axis`` on."""
    if not -len(shape) <= axis < len(shape):
        raise ValueError(f"axis {axis} out of range for X of shape {tuple(shape)}")
    axis %= len(shape)
    rows = D = 1
    for n in shape[:axis]:
        rows *= n
    for n in shape[axis:]:
        D *= n
    return rows, D, tuple(shape[axis:]), tuple(shape[:axis]) + (1,) * (len(shape) - axis)


def gs_layer_norm(X, Scale, B=None, axis=-1, epsilon=1e-5, out=None):
    """LayerNormalization of X over its axes from ``axis`` on: (Y, Mean, InvStdDev).  Scale and B
    have the shape of the normalised axes; Mean and InvStdDev are float32 with X's leading axes
    and ones in the place of the normalised ones (NaN where those hold no element)."""
    rows, D, inner, kept = _norm_dims(X.shape, operator.index(axis))
    _check_input(X)
    _check_like(X, "Scale", Scale, inner)
    if B is not None:
        _check_like(X, "B", B, inner)
    h = _host()
    empty, device = h.torch.empty, X.device
    if out is None:
        out = empty(X.shape, dtype=X.dtype, device=device)
    else:
        _check_like(X, "out", out, X.shape)
    mean = empty(kept, dtype=h.torch.float32, device=device)
    inv = empty(kept, dtype=h.torch.float32, device=device)
    status = h.lib.gs_layer_norm(X.data_ptr(), Scale.data_ptr(), _p(B), rows, D, h.codes[X.dtype],
                                 epsilon, out.data_ptr(), mean.data_ptr(), inv.data_ptr(),
                                 h.stream(device.index))
    if status:
        raise GsError(status, "gs_layer_norm")
    if D == 0:   # the call writes nothing; the mean of no element
        mean.fill_(float("nan"))
        inv.fill_(float("nan"))
    return out, mean, inv


@functools.lru_cache(maxsize=256)
def gs_layer_norm_backward_workspace_size(rows, D):
    """Workspace bytes gs_layer_norm_backward needs."""
    n = ctypes.c_size_t(0)
    _ok(load_library().gs_layer_norm_backward_workspace_size(rows, D, ctypes.byref(n)),
        "gs_layer_norm_backward_workspace_size")
    return int(n.value)


def gs_layer_norm_backward(dY, X, Scale, Mean, InvStdDev, axis=-1, workspace="auto"):
    """Gradient of gs_layer_norm: (dX, dScale, dB).  ``workspace``: "auto", or a device tensor of
    at least gs_layer_norm_backward_workspace_size bytes."""
    rows, D, inner, kept = _norm_dims(X.shape, operator.index(axis))
    _check_input(X)
    _check_like(X, "dY", dY, X.shape)
    _check_like(X, "Scale", Scale, inner)
    _check_f32(Mean, kept, "Mean", X)
    _check_f32(InvStdDev, kept, "InvStdDev", X)
    h = _host()
    empty, device, dt = h.torch.empty, X.device, X.dtype
    dX = empty(X.shape, dtype=dt, device=device)
    dScale = empty(inner, dtype=dt, device=device)
    dB = empty(inner, dtype=dt, device=device)
    ws, have, _keep = _scratch(workspace, gs_layer_norm_backward_workspace_size(rows, D), X)
    status = h.lib.gs_layer_norm_backward(
        dY.data_ptr(), X.data_ptr(), Scale.data_ptr(), Mean.data_ptr(), InvStdDev.data_ptr(), rows,
        D, h.codes[dt], ws, have, dX.data_ptr(), dScale.data_ptr(), dB.data_ptr(),
        h.stream(device.index))
    if status:
        raise GsError(status, "gs_layer_norm_backward")
    return dX, dScale, dB


# ------------------------------------------------------------------ dropout

def gs_dropout(X, ratio=0.5, seed=0, offset=0, residual=None, out=None):
    """residual + dropout(X) with the mask of (seed, offset), which is stored nowhere.  The
    gradient with respect to X is ``gs_dropout(dY, ratio, seed, offset)``.  ``out`` may be X or
    residual itself."""
    _check_input(X)
    if residual is not None:
        _check_like(X, "residual", residual, X.shape)
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 64:
        raise ValueError("seed and offset are unsigned 64-bit numbers")
    h = _host()
    if out is None:
        out = h.torch.empty(X.shape, dtype=X.dtype, device=X.device)
    else:
        _check_like(X, "out", out, X.shape)
    status = h.lib.gs_dropout(X.data_ptr(), _p(residual), X.numel(), h.codes[X.dtype], ratio, seed,
                              offset, out.data_ptr(), h.stream(X.device.index))
    if status:
        raise GsError(status, "gs_dropout")
    return out


# ------------------------------------------------------------------ attention

def gs_relative_buckets(q_extent, k_extent, num_buckets=0, max_distance=128, causal=False,
                        q_origin=(0, 0), device="cuda"):
    """Bucket map for gs_attention: (int32 tensor (Hq+Hk-1, Wq+Wk-1) on ``device``, rows of the
    bias table).  ``num_buckets`` 0 gives every relative position a row of its own."""
    torch = _torch()
    rows, cols = q_extent[0] + k_extent[0] - 1, q_extent[1] + k_extent[1] - 1
    m = torch.empty((max(rows, 0), max(cols, 0)), dtype=torch.int32)
    count = ctypes.c_int64(0)
    _ok(load_library().gs_relative_buckets(
        _i64(q_extent), _i64(k_extent), _i64(q_origin), int(num_buckets), int(max_distance),
        int(causal), ctypes.cast(m.data_ptr(), ctypes.POINTER(ctypes.c_int32)),
        ctypes.byref(count)), "gs_relative_buckets")
    return m.to(device), int(count.value)


def _attention_attrs(Q, K, V, table, q_extent, k_extent, scale):
    """AttentionAttrs of tensors whose shapes and strides fit together."""
    for t, what in ((Q, "Q"), (K, "K"), (V, "V")):
        if t.dim() != 4:
            raise ValueError(f"{what} must be (N, L, H, D), got {tuple(t.shape)}")
        if t.stride(3) != 1 and t.shape[3] != 1:
            raise ValueError(f"the last axis of {what} must be contiguous")
    N, Lq, H, D = Q.shape
    if D == 0:
        raise ValueError(f"heads of width 0: Q is {tuple(Q.shape)}")
    Lk = K.shape[1]
    if K.shape != (N, Lk, H, D):
        _shape_error("K", K.shape, (N, Lk, H, D))
    if V.shape != K.shape:
        _shape_error("V", V.shape, K.shape)
    q_extent = (1, Lq) if q_extent is None else q_extent
    k_extent = (1, Lk) if k_extent is None else k_extent
    if len(q_extent) != 2 or len(k_extent) != 2:
        raise ValueError(f"an extent is (rows, columns), got {q_extent} and {k_extent}")
    if q_extent[0] * q_extent[1] != Lq or k_extent[0] * k_extent[1] != Lk:
        raise ValueError(f"extents {q_extent} and {k_extent} do not hold {Lq} and {Lk} tokens")
    nb = 0
    if table is not None:
        if table.dim() != 2 or table.shape[1] != H:
            raise ValueError(f"table must be (buckets, H={H}), got {tuple(table.shape)}")
        nb = table.shape[0]
    i3, i2 = ctypes.c_int64 * 3, ctypes.c_int64 * 2
    return AttentionAttrs(N, H, D, i2(*q_extent), i2(*k_extent), i3(*Q.stride()[:3]),
                          i3(*K.stride()[:3]), i3(*V.stride()[:3]), nb,
                          D ** -0.5 if scale is None else scale)


class _Plan:
    """What a call's shapes, strides and dtype alone decide: the C attributes and the workspace
    sizes.  Kept per signature, since building and checking them takes longer than a launch."""

    def __init__(self, Q, K, V, table, q_extent, k_extent, scale):
        self.attrs = _attention_attrs(Q, K, V, table, q_extent, k_extent, scale)
        self.ref = ctypes.byref(self.attrs)
        if Q.dtype not in _host().codes:
            raise TypeError(f"unsupported dtype {Q.dtype}")
        self.code = _host().codes[Q.dtype]
        at = self.attrs
        self.lse_shape = (at.N, at.H, Q.shape[1])
        self.entries = ((at.q_extent[0] + at.k_extent[0] - 1)
                        * (at.q_extent[1] + at.k_extent[1] - 1) if Q.shape[1] and K.shape[1] else 0)
        self._bytes = {}

    def workspace(self, backward):
        if backward not in self._bytes:
            self._bytes[backward] = gs_attention_workspace_size(self.attrs, self.code, backward)
        return self._bytes[backward]


_PLANS = {}
_MOST_PLANS = 256


def _extent(e):
    """A grid's extent as a tuple of whole numbers; None stays None."""
    return None if e is None else tuple(map(operator.index, e))


def _plan(Q, K, V, table, buckets, q_extent, k_extent, k_len, scale):
    torch = _host().torch
    if scale is not None:
        scale = float(scale)   # a plan holds numbers: a tensor would be known by its identity
    q_extent, k_extent = _extent(q_extent), _extent(k_extent)
    key = (Q.shape, Q.stride(), K.shape, K.stride(), V.shape, V.stride(), Q.dtype,
           None if table is None else table.shape, q_extent, k_extent, scale)
    plan = _PLANS.get(key)
    if plan is None:
        plan = _Plan(Q, K, V, table, q_extent, k_extent, scale)
        if len(_PLANS) >= _MOST_PLANS:
            _PLANS.clear()
        _PLANS[key] = plan
    device = Q.device
    if device.type != "cuda":
        raise ValueError("libgs takes CUDA tensors")
    if (K.dtype != Q.dtype or V.dtype != Q.dtype or K.device != device or V.device != device
            or (table is not None and (table.dtype != Q.dtype or table.device != device))):
        raise ValueError("all tensors of one call share dtype and device")
    if table is None:
        if buckets is not None:
            raise ValueError("table and buckets go together")
    elif buckets is None:
        raise ValueError("table and buckets go together")
    elif (buckets.dtype != torch.int32 or buckets.device != device
          or not buckets.is_contiguous() or not table.is_contiguous()
          or (plan.entries and buckets.numel() != plan.entries)):
        raise ValueError(f"table must be contiguous, buckets a contiguous int32 tensor of "
                         f"{plan.entries} entries on the inputs' device")
    if k_len is not None and (k_len.dtype != torch.int32 or k_len.device != device
                              or not k_len.is_contiguous() or k_len.shape != Q.shape[:1]):
        raise ValueError(f"k_len must be a contiguous int32 tensor of N={Q.shape[0]} entries on "
                         f"the inputs' device")
    return plan


def gs_attention_workspace_size(attrs, dtype_code, backward=False):
    """Workspace bytes gs_attention (or gs_attention_backward) needs for an AttentionAttrs."""
    n = ctypes.c_size_t(0)
    name = "gs_attention_backward_workspace_size" if backward else "gs_attention_workspace_size"
    _ok(getattr(load_library(), name)(ctypes.byref(attrs), dtype_code, ctypes.byref(n)), name)
    return n.value


def gs_attention_backward_workspace_size(attrs, dtype_code):
    """Workspace bytes gs_attention_backward needs for an AttentionAttrs."""
    return gs_attention_workspace_size(attrs, dtype_code, True)


def gs_attention(Q, K, V, table=None, buckets=None, q_extent=None, k_extent=None, k_len=None,
                 scale=None, out=None, workspace="auto"):
    """softmax(scale Q K^T + table[bucket]) V over grids of tokens: (O, LSE).

    Q (N, Lq, H, D), K and V (N, Lk, H, D), any strides with a contiguous last axis; ``table``
    (buckets, H) and ``buckets`` (int32, see gs_relative_buckets) name each pair's bias;
    ``q_extent`` / ``k_extent`` are the tokens' grids (default (1, L)); ``k_len`` (N) int32 masks
    the keys from there on; ``scale`` is a number, read at every call (a one-element
    tensor's value as well), and defaults to 1 / sqrt(D).  O is dense (N, Lq, H, D), LSE
    float32 (N, H, Lq)."""
    plan = _plan(Q, K, V, table, buckets, q_extent, k_extent, k_len, scale)
    h = _host()
    empty, device = h.torch.empty, Q.device
    if out is None:
        out = empty(Q.shape, dtype=Q.dtype, device=device)
    else:
        _check_like(Q, "out", out, Q.shape)
    lse = empty(plan.lse_shape, dtype=h.torch.float32, device=device)
    ws, have, _keep = _scratch(workspace, plan.workspace(False), Q)
    status = h.lib.gs_attention(Q.data_ptr(), K.data_ptr(), V.data_ptr(), _p(table), _p(buckets),
                                _p(k_len), plan.ref, plan.code, ws, have, out.data_ptr(),
                                lse.data_ptr(), h.stream(device.index))
    if status:
        raise GsError(status, "gs_attention")
    return out, lse


def gs_attention_backward(dO, Q, K, V, O, LSE, table=None, buckets=None, q_extent=None,
                          k_extent=None, k_len=None, scale=None, workspace="auto"):
    """Gradient of gs_attention: [dQ, dK, dV, dTable] (the first three without a table); dQ, dK
    and dV are dense (N, L, H, D)."""
    plan = _plan(Q, K, V, table, buckets, q_extent, k_extent, k_len, scale)
    _check_like(Q, "dO", dO, Q.shape)
    _check_like(Q, "O", O, Q.shape)
    _check_f32(LSE, plan.lse_shape, "LSE", Q)
    h = _host()
    empty, device, dt = h.torch.empty, Q.device, Q.dtype
    made = [empty(Q.shape, dtype=dt, device=device), empty(K.shape, dtype=dt, device=device),
            empty(K.shape, dtype=dt, device=device)]
    if table is not None:
        made.append(empty(table.shape, dtype=dt, device=device))
    ws, have, _keep = _scratch(workspace, plan.workspace(True), Q)
    status = h.lib.gs_attention_backward(
        dO.data_ptr(), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(),
        _p(table), _p(buckets), _p(k_len), plan.ref, plan.code, ws, have, made[0].data_ptr(),
        made[1].data_ptr(), made[2].data_ptr(), made[3].data_ptr() if table is not None else None,
        h.stream(device.index))
    if status:
        raise GsError(status, "gs_attention_backward")
    return made
