"""Refusals and host logic of the feed-forward entry points: no GPU needed, since bad arguments
are refused before anything is enqueued."""
import ctypes
import math

import pytest
import torch

import spatial_transformer_sampling_gb300 as gs
from spatial_transformer_sampling_gb300 import build as gsbuild

FAKE = 0x10000   # a non-null, aligned pointer value; never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    gsbuild.build()
    return gs.load_library()


def _bytes(f, *args):
    n = ctypes.c_size_t(0)
    assert f(*args, ctypes.byref(n)) == 0
    return n.value


SIZES = [(dict(dt=3), 4), (dict(act=6), 5), (dict(act=-1), 5), (dict(rows=-1), 3), (dict(D=0), 3),
         (dict(D=-3), 3), (dict(D=(1 << 20) + 1), 3), (dict(F=-1), 3), (dict(F=(1 << 20) + 1), 3),
         (dict(rows=1 << 31), 3), (dict(rows=(1 << 31) - 1, D=1 << 10), 3)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(X=None), 1), (dict(Wg=None), 1), (dict(Wu=None), 1), (dict(H=None), 1), (dict(bg=FAKE), 1),
    (dict(bu=FAKE), 1), (dict(G=FAKE), 1), (dict(U=FAKE), 1), (dict(X=FAKE + 2), 6),
    (dict(Wu=FAKE + 1, dt=2), 6), (dict(H=FAKE + 2), 6), (dict(G=FAKE + 2, U=FAKE), 6),
    (dict(rows=0, X=None), 0), (dict(F=0, H=None), 0)])
def test_gated_linear_refuses(L, kw, status):
    a = dict(X=FAKE, Wg=FAKE, Wu=FAKE, bg=None, bu=None, rows=300, D=24, F=40, act=0, dt=0, ws=FAKE,
             have=1 << 30, H=FAKE, G=None, U=None)
    a.update(kw)
    assert L.gs_gated_linear(*(a[k] for k in ("X", "Wg", "Wu", "bg", "bu", "rows", "D", "F", "act",
                                              "dt", "ws", "have", "H", "G", "U")), None) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict([(k, None)]), 1) for k in ("dH", "X", "Wg", "Wu", "G", "U", "dX", "dWg", "dWu")] + [
    (dict(dbg=FAKE), 1), (dict(dbu=FAKE), 1), (dict(dX=FAKE + 2), 6), (dict(G=FAKE + 1, dt=1), 6),
    (dict(dbg=FAKE + 2, dbu=FAKE), 6), (dict(ws=None), 1), (dict(ws=FAKE + 16), 6),
    (dict(have=1024), 3)])
def test_gated_linear_backward_refuses(L, kw, status):
    a = dict(dH=FAKE, X=FAKE, Wg=FAKE, Wu=FAKE, G=FAKE, U=FAKE, rows=300, D=24, F=40, act=0, dt=0,
             ws=FAKE, have=1 << 30, dX=FAKE, dWg=FAKE, dWu=FAKE, dbg=None, dbu=None)
    a.update(kw)
    assert L.gs_gated_linear_backward(
        *(a[k] for k in ("dH", "X", "Wg", "Wu", "G", "U", "rows", "D", "F", "act", "dt", "ws", "have",
                         "dX", "dWg", "dWu", "dbg", "dbu")), None) == status


def test_gated_linear_workspace_queries(L):
    n = ctypes.c_size_t(7)
    for f in (L.gs_gated_linear_workspace_size, L.gs_gated_linear_backward_workspace_size):
        assert f(4, 8, 8, 0, None) == 1
        assert f(-1, 8, 8, 0, ctypes.byref(n)) == 3 and n.value == 0
        assert f(4, 8, 8, 9, ctypes.byref(n)) == 4
        assert _bytes(f, 0, 8, 8, 0) == 0 and _bytes(f, 4, 8, 0, 0) == 0
        for dt in range(3):
            for rows in (1, 77, 5000):
                assert _bytes(f, rows, 33, 50, dt) % 256 == 0
    # few rows are multiplied where they lie; rows too long for that are not
    for dt in range(3):
        assert _bytes(L.gs_gated_linear_workspace_size, 32, 33, 50, dt) == 0
        assert _bytes(L.gs_gated_linear_workspace_size, 33, 33, 50, dt) > 0
        assert _bytes(L.gs_gated_linear_workspace_size, 16, 33, 5000, dt) == 0
        assert _bytes(L.gs_gated_linear_workspace_size, 17, 33, 5000, dt) > 0
    assert _bytes(L.gs_gated_linear_workspace_size, 32, 262144 + 1, 50, 0) == 0
    assert _bytes(L.gs_gated_linear_workspace_size, 32, 262144 + 1, 50, 1) > 0
    # dG and dU at least
    assert _bytes(L.gs_gated_linear_backward_workspace_size, 1000, 64, 128, 1) >= 2 * 1000 * 128 * 2


def _attrs(kw):
    a = dict(rows=60, D=24, groups=0, kind=0, alpha=1.0, epsilon=1e-5)
    a.update({k: kw.pop(k) for k in list(kw) if k in a})
    return gs.ResidualNormAttrs(a["rows"], a["D"], a["groups"], a["kind"], a["alpha"], a["epsilon"])


FORMS = [(dict(dt=5), 4), (dict(kind=2), 5), (dict(alpha=math.inf), 5), (dict(alpha=math.nan), 5),
         (dict(epsilon=-1.0), 5), (dict(epsilon=math.nan), 5), (dict(epsilon=math.inf), 5),
         (dict(rows=-1), 3), (dict(D=-1), 3), (dict(D=(1 << 20) + 1), 3), (dict(rows=1 << 31), 3),
         (dict(groups=-1), 3), (dict(groups=7), 3), (dict(groups=120), 3), (dict(groups=2), 1),
         (dict(D=0), 0)]


@pytest.mark.parametrize("kw,status", FORMS + [
    (dict([(k, None)]), 1) for k in ("X", "Z", "Scale", "S", "Y")] + [
    (dict(gate=FAKE), 3), (dict(z_B=FAKE), 1), (dict(X=FAKE + 2), 6), (dict(Y=FAKE + 1, dt=1), 6),
    (dict(Stats=FAKE + 8), 6), (dict(rows=0, X=None), 0)])
def test_residual_norm_refuses(L, kw, status):
    kw = dict(kw)
    at = _attrs(kw)
    a = dict(X=FAKE, Z=FAKE, gate=None, z_scale=None, z_B=None, Scale=FAKE, B=None, dt=0, S=FAKE,
             Y=FAKE, Stats=FAKE)
    a.update(kw)
    assert L.gs_residual_norm(*(a[k] for k in ("X", "Z", "gate", "z_scale", "z_B", "Scale", "B")),
                              ctypes.byref(at), a["dt"], a["S"], a["Y"], a["Stats"], None) == status


@pytest.mark.parametrize("kw,status", FORMS + [
    (dict([(k, None)]), 1) for k in ("dY", "S", "Z", "Stats", "Scale", "dX", "dZ")] + [
    (dict(dgate=FAKE), 3), (dict(dz_scale=FAKE), 1), (dict(dz_B=FAKE), 1), (dict(z_B=FAKE), 1),
    (dict(groups=2, gate=FAKE), 1), (dict(dS=FAKE + 2), 6), (dict(Stats=FAKE + 4), 6),
    (dict(ws=None), 1), (dict(ws=FAKE + 128), 6), (dict(have=16), 3)])
def test_residual_norm_backward_refuses(L, kw, status):
    kw = dict(kw)
    at = _attrs(kw)
    names = ("dS", "dY", "S", "Z", "Stats", "gate", "z_scale", "z_B", "Scale")
    outs = ("dX", "dZ", "dgate", "dz_scale", "dz_B", "dScale", "dB")
    a = dict.fromkeys(names + outs, FAKE)
    a.update(dict.fromkeys(("gate", "z_scale", "z_B", "dgate", "dz_scale", "dz_B")), dt=0, ws=FAKE,
             have=1 << 30)
    a.update(kw)
    assert L.gs_residual_norm_backward(*(a[k] for k in names), ctypes.byref(at), a["dt"], a["ws"],
                                       a["have"], *(a[k] for k in outs), None) == status


def test_residual_norm_workspace_queries(L):
    f, n = L.gs_residual_norm_backward_workspace_size, ctypes.c_size_t(7)
    at = gs.ResidualNormAttrs
    assert f(None, 0, ctypes.byref(n)) == 1 and f(ctypes.byref(at(4, 8, 0, 0, 1.0, 0.0)), 0, None) == 1
    assert f(ctypes.byref(at(4, -8, 0, 0, 1.0, 0.0)), 0, ctypes.byref(n)) == 3 and n.value == 0
    assert _bytes(f, ctypes.byref(at(0, 8, 0, 0, 1.0, 0.0)), 0) == 0
    assert _bytes(f, ctypes.byref(at(4, 0, 0, 0, 1.0, 0.0)), 0) == 0
    for groups in (0, 1, 5, 100, 50000, 100000):
        for D in (8, 771, 9000):
            b = _bytes(f, ctypes.byref(at(100000, D, groups, 0, 1.0, 0.0)), 1)
            # a few sums per SM and column; the gate's are in the output where there are many
            assert 0 < b <= (1 << 27) + 100000 * 8, (groups, D, b)


def test_binding_refuses_what_does_not_fit():
    X, W = torch.zeros(4, 8), torch.zeros(16, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gs.gs_gated_linear(X, W, W)
    with pytest.raises(ValueError, match="activation"):
        gs.gs_gated_linear(X, W, W, activation="swish")
    with pytest.raises(ValueError, match="CUDA"):
        gs.gs_residual_norm(X, X, X[0])
    with pytest.raises(ValueError, match="CUDA"):
        gs.gs_residual_norm_backward(X, X, X, X, X, X[0])
