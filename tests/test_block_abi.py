"""Refusals and host logic of the transformer-block entry points: no GPU needed, since bad
arguments are refused before anything is enqueued."""
import ctypes
import math

import pytest
import torch

import block_reference as ref
import spatial_transformer_sampling_gb300 as gs
from spatial_transformer_sampling_gb300 import build as gsbuild

FAKE = 0x10000   # a non-null, aligned pointer value; never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    gsbuild.build()
    return gs.load_library()


# ------------------------------------------------------------------ layer norm

@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), 4), (dict(rows=-1), 3), (dict(D=-1), 3), (dict(D=(1 << 20) + 1), 3),
    (dict(rows=1 << 31), 3), (dict(eps=-1e-5), 5), (dict(eps=math.nan), 5),
    (dict(eps=math.inf), 5), (dict(X=None), 1), (dict(S=None), 1), (dict(Y=None), 1),
    (dict(X=FAKE + 2), 6), (dict(dt=2, Y=FAKE + 1), 6), (dict(B=FAKE + 3), 6),
    (dict(M=FAKE + 2), 6), (dict(rows=0, X=None, Y=None), 0), (dict(D=0, X=None), 0),
])
def test_layer_norm_refuses(L, kw, status):
    a = dict(X=FAKE, S=FAKE, B=None, rows=4, D=8, dt=0, eps=1e-5, Y=FAKE, M=FAKE, I=FAKE)
    a.update(kw)
    assert L.gs_layer_norm(a["X"], a["S"], a["B"], a["rows"], a["D"], a["dt"], a["eps"], a["Y"],
                           a["M"], a["I"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=-1), 4), (dict(rows=-1), 3), (dict(dY=None), 1), (dict(M=None), 1), (dict(dX=None), 1),
    (dict(ws=None, have=0), 1), (dict(have=16), 3), (dict(ws=FAKE + 4), 6), (dict(dS=FAKE + 2), 6),
    (dict(D=0), 0),
])
def test_layer_norm_backward_refuses(L, kw, status):
    n = ctypes.c_size_t(0)
    assert L.gs_layer_norm_backward_workspace_size(100, 8, ctypes.byref(n)) == 0 and n.value > 0
    a = dict(dY=FAKE, X=FAKE, S=FAKE, M=FAKE, I=FAKE, rows=100, D=8, dt=0, ws=FAKE, have=n.value,
             dX=FAKE, dS=FAKE, dB=FAKE)
    a.update(kw)
    assert L.gs_layer_norm_backward(a["dY"], a["X"], a["S"], a["M"], a["I"], a["rows"], a["D"],
                                    a["dt"], a["ws"], a["have"], a["dX"], a["dS"], a["dB"],
                                    None) == status


def test_layer_norm_workspace_query(L):
    n = ctypes.c_size_t(7)
    assert L.gs_layer_norm_backward_workspace_size(10, 8, None) == 1
    assert L.gs_layer_norm_backward_workspace_size(-1, 8, ctypes.byref(n)) == 3 and n.value == 0
    assert L.gs_layer_norm_backward_workspace_size(0, 8, ctypes.byref(n)) == 0 and n.value == 0


# ------------------------------------------------------------------ dropout

@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), 4), (dict(n=-1), 3), (dict(n=(1 << 40) + 1), 3), (dict(ratio=1.0), 5),
    (dict(ratio=-0.1), 5), (dict(ratio=math.nan), 5), (dict(X=None), 1), (dict(Y=None), 1),
    (dict(X=FAKE + 1), 6), (dict(R=FAKE + 2), 6), (dict(n=0, X=None, Y=None), 0),
])
def test_dropout_refuses(L, kw, status):
    a = dict(X=FAKE, R=None, n=10, dt=0, ratio=0.5, Y=FAKE)
    a.update(kw)
    assert L.gs_dropout(a["X"], a["R"], a["n"], a["dt"], a["ratio"], 1, 2, a["Y"], None) == status


def test_generator_against_published_vectors():
    # Philox4x32-10 known answers of the method's authors (counter and key all zeros, all ones)
    assert ref.philox_words(4, 0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


# ------------------------------------------------------------------ attention

def _attrs(N=2, H=3, D=64, q=(4, 5), k=(4, 5), qs=None, ks=None, vs=None, nb=10, scale=0.125):
    i3, i2 = ctypes.c_int64 * 3, ctypes.c_int64 * 2
    d = (q[0] * q[1] * H * D, H * D, D)
    return gs.AttentionAttrs(N, H, D, i2(*q), i2(*k), i3(*(qs or d)), i3(*(ks or d)),
                             i3(*(vs or d)), nb, scale)


BAD_SHAPES = [
    (dict(N=-1), 3), (dict(H=-1), 3), (dict(D=0), 3), (dict(D=129), 3), (dict(q=(-1, 5)), 3),
    (dict(k=(4, -5)), 3), (dict(q=(1 << 20, 1 << 20)), 3), (dict(N=1 << 20, H=1 << 20), 3),
    (dict(N=1 << 16, q=(1, 1 << 16)), 3), (dict(qs=(1, -1, 1)), 3), (dict(vs=(-1, 1, 1)), 3),
    (dict(nb=-1), 3), (dict(nb=1 << 31), 3), (dict(q=(1, 1 << 23), k=(1, 1 << 24)), 3),
    (dict(scale=math.nan), 5), (dict(scale=math.inf), 5),
]


@pytest.mark.parametrize("kw,status", BAD_SHAPES)
def test_attention_refuses_shapes(L, kw, status):
    at, n = _attrs(**kw), ctypes.c_size_t(5)
    for f in (L.gs_attention_workspace_size, L.gs_attention_backward_workspace_size):
        assert f(ctypes.byref(at), 0, ctypes.byref(n)) == status and n.value == 0
    assert L.gs_attention(FAKE, FAKE, FAKE, FAKE, FAKE, None, ctypes.byref(at), 0, FAKE, 1 << 30,
                          FAKE, FAKE, None) == status
    assert L.gs_attention_backward(*[FAKE] * 8, None, ctypes.byref(at), 0, FAKE, 1 << 30,
                                   *[FAKE] * 4, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=5), 4), (dict(at=None), 1), (dict(Q=None), 1), (dict(K=None), 1), (dict(V=None), 1),
    (dict(O=None), 1), (dict(table=None), 1), (dict(buckets=None), 1), (dict(Q=FAKE + 2), 6),
    (dict(dt=1, O=FAKE + 1), 6), (dict(buckets=FAKE + 2), 6), (dict(k_len=FAKE + 1), 6),
    (dict(lse=FAKE + 2), 6), (dict(ws=None, have=0), 1), (dict(ws=FAKE + 16), 6),
    (dict(have=8), 3), (dict(at=_attrs(nb=0)), 3), (dict(at=_attrs(N=0), Q=None, O=None), 0),
    (dict(at=_attrs(q=(0, 5)), Q=None, O=None), 0),
])
def test_attention_refuses_arguments(L, kw, status):
    a = dict(Q=FAKE, K=FAKE, V=FAKE, table=FAKE, buckets=FAKE, k_len=None, at=_attrs(), dt=0,
             ws=FAKE, have=1 << 30, O=FAKE, lse=FAKE)
    a.update(kw)
    at = ctypes.byref(a["at"]) if a["at"] is not None else None
    assert L.gs_attention(a["Q"], a["K"], a["V"], a["table"], a["buckets"], a["k_len"], at,
                          a["dt"], a["ws"], a["have"], a["O"], a["lse"], None) == status


@pytest.mark.parametrize("which,status", [(i, 1) for i in range(8)] + [(13, 1), (14, 1), (15, 1),
                                                                       (16, 1)])
def test_attention_backward_needs_every_pointer(L, which, status):
    at = _attrs()
    a = [FAKE] * 8 + [None, ctypes.byref(at), 0, FAKE, 1 << 30] + [FAKE] * 4 + [None]
    a[which] = None
    assert L.gs_attention_backward(*a) == status
    a[which] = FAKE + 1   # and aligned ones
    assert L.gs_attention_backward(*a) == 6


def test_attention_workspace_queries(L):
    n = ctypes.c_size_t(0)
    at = _attrs()
    assert L.gs_attention_workspace_size(ctypes.byref(at), 0, None) == 1
    assert L.gs_attention_workspace_size(None, 0, ctypes.byref(n)) == 1
    assert L.gs_attention_workspace_size(ctypes.byref(at), 9, ctypes.byref(n)) == 4
    empty = _attrs(N=0)
    assert L.gs_attention_backward_workspace_size(ctypes.byref(empty), 0, ctypes.byref(n)) == 0
    assert n.value == 0


# ------------------------------------------------------------------ bucket maps

def _plain_axis(offset, num, far):
    m, e = num // 2, num // 4
    d = abs(offset)
    starts = [e * (far / e) ** (k / (m - e)) for k in range(m - e)]
    b = d if d < e else e + max(k for k in range(m - e) if d >= math.ceil(starts[k] - 1e-9))
    return b + (m if offset < 0 else 0)


@pytest.mark.parametrize("q,k,num,far,origin", [
    ((1, 9), (1, 9), 8, 16, (0, 0)), ((1, 1), (1, 300), 32, 128, (0, 299)),
    ((5, 7), (6, 4), 8, 5, (1, 2)), ((9, 1), (9, 1), 6, 20, (0, 0)), ((1, 50), (1, 70), 4, 3, (0, 20)),
    ((1, 1), (1, 1), 8, 9, (0, 0)),
])
def test_relative_buckets_follow_their_definition(L, q, k, num, far, origin):
    m, count = gs.gs_relative_buckets(q, k, num, far, False, origin, device="cpu")
    rows, cols = q[0] + k[0] - 1, q[1] + k[1] - 1
    assert tuple(m.shape) == (rows, cols)
    axes = [n for n in (rows, cols) if n > 1]
    assert count == num ** len(axes)
    for r in range(rows):
        for c in range(cols):
            dy, dx = r - (k[0] - 1) + origin[0], c - (k[1] - 1) + origin[1]
            want = 0
            if rows > 1:
                want = _plain_axis(dy, num, far)
            if cols > 1:
                want = want * num * (rows > 1) + _plain_axis(dx, num, far)
            assert m[r, c].item() == want


def test_relative_buckets_one_per_offset_and_causal(L):
    m, count = gs.gs_relative_buckets((3, 4), (3, 4), device="cpu")
    assert count == 35 and torch.equal(m.flatten(), torch.arange(35, dtype=torch.int32))
    m, count = gs.gs_relative_buckets((1, 4), (1, 6), 0, causal=True, q_origin=(0, 2), device="cpu")
    off = torch.arange(9) - 5 + 2
    assert torch.equal(m[0] < 0, off < 0) and count == 9


@pytest.mark.parametrize("kw,status", [
    (dict(num_buckets=3), 5), (dict(num_buckets=2), 5), (dict(num_buckets=7), 5),
    (dict(num_buckets=8, max_distance=2), 5), (dict(num_buckets=-4), 5),
    (dict(q=(2, 3), causal=True), 9), (dict(q=(-1, 3)), 3), (dict(q=(1, 1 << 24), fake=True), 3),
])
def test_relative_buckets_refuse(L, kw, status):
    a = dict(q=(1, 3), k=(1, 3), num_buckets=8, max_distance=16, causal=False)
    a.update(kw)
    i2, n = ctypes.c_int64 * 2, ctypes.c_int64(0)
    buf = (ctypes.c_int32 * 64)()
    assert L.gs_relative_buckets(i2(*a["q"]), i2(*a["k"]), None, a["num_buckets"],
                                 a["max_distance"], int(a["causal"]), buf,
                                 ctypes.byref(n)) == status
    assert L.gs_relative_buckets(None, i2(1, 1), None, 0, 0, 0, buf, ctypes.byref(n)) == 1


# ------------------------------------------------------------------ the binding's own checks

def test_binding_refuses_mismatched_tensors():
    t = torch.zeros((2, 6, 3, 8))
    with pytest.raises(ValueError):
        gs.gs_attention(t, t, t)                                        # not on a GPU
    with pytest.raises(ValueError):
        gs.gs_attention(t, t[:, :5], t)                                  # V is not K's shape
    with pytest.raises(ValueError):
        gs.gs_attention(t, t.transpose(2, 3), t)
    with pytest.raises(ValueError):
        gs.gs_layer_norm(t, torch.ones(8))                               # not on a GPU
    with pytest.raises(ValueError):
        gs.gs_layer_norm(t, torch.ones(8), axis=4)
    with pytest.raises(ValueError):
        gs.gs_dropout(t, 0.5)
    with pytest.raises(ValueError):
        gs.gs_attention_backward(t, t, t, t, t, t)
