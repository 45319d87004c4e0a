"""Every shape of the residual norm's and the gated projections' kernels that the library holds is
one that some width and alignment takes, and none is missing."""
import re
import shutil
import subprocess

import pytest

from spatial_transformer_sampling_gb300 import build as gsbuild

RUN = {"float": 4, "__half": 8, "__nv_bfloat16": 8}   # elements of 16 bytes
SIZE = {"float": 4, "__half": 2, "__nv_bfloat16": 2}
ON_CHIP, STAGED, MOST = 8192, 4096, 1 << 20


@pytest.fixture(scope="module")
def held():
    """{kernel: set of its template arguments}, as the symbol table names them."""
    if not shutil.which("nm"):
        pytest.skip("no nm")
    names = subprocess.run(["nm", "-C", "--defined-only", gsbuild.build()], check=True,
                           capture_output=True, text=True).stdout
    out = {}
    for name, args in re.findall(r"\bvoid gs::(\w+_kernel)<([^>]*)>\(", names):
        out.setdefault(name, set()).add(tuple(a.strip() for a in args.split(",")))
    return out


def _runs(T):
    """Elements per access, and the widths that may come with it."""
    return [(1, 1), (2, 2), (RUN[T], RUN[T])]


def _first(table, D):
    return next(shape for shape in table if D <= shape[-2] * shape[-1])


def _forward(T):
    """(V, L, NV) of the widths up to ON_CHIP."""
    single = [(8, 4), (8, 6), (8, 8), (16, 6), (16, 8), (32, 6), (32, 8), (32, 12), (32, 16), (64, 12),
              (64, 16), (128, 12), (128, 16), (256, 12), (256, 16), (256, 24), (256, 32)]
    runs = [(4, 1), (8, 1), (16, 1), (32, 1), (32, 2), (32, 3), (32, 4), (64, 3), (64, 4), (128, 3),
            (128, 4), (256, 3), (256, 4), (256, 6), (256, 8)]
    for V, step in _runs(T):
        for D in range(step, ON_CHIP + 1, step):
            if V <= 2:
                L, N = _first(single, D)
                yield V, L, N // V
            else:
                yield (V,) + _first(runs, D // V)


def _backward(T, more):
    """(staged, V, L, NV) of the widths that are not read twice."""
    narrow = [(0, 8, 2), (0, 8, 3), (0, 8, 4), (0, 8, 6), (0, 16, 4), (0, 16, 6), (0, 32, 4), (0, 32, 5),
              (1, 32, 6), (1, 32, 8), (1, 64, 6), (1, 64, 8), (1, 128, 6), (1, 128, 8), (1, 256, 6),
              (1, 256, 8), (1, 512, 6), (1, 512, 8), (0, 512, 16)]
    for V, step in _runs(T):
        few = [(0, L, V) for L in (4, 8, 16, 32)]
        table = ([s for s in narrow if s[2] % V == 0] if V <= 2 else
                 few + [(1, L, 8) for L in (32, 64, 128, 256, 512)] + [(0, 512, 16)])
        for D in range(step, (STAGED if more else ON_CHIP) + 1, step):
            staged, L, N = _first(table, D)
            yield staged, V, L, N // V


def _named(T, shape, *flags):
    return (T,) + tuple(str(n) for n in shape) + tuple("true" if f else "false" for f in flags)


def test_residual_norm(held):
    forward, wide, back, staged = set(), set(), set(), set()
    for T in RUN:
        for post in (False, True):
            forward |= {_named(T, s, post) for s in _forward(T)}
            for gate in (False, True):
                for s, *shape in _backward(T, post or gate):
                    (staged if s else back).add(_named(T, shape, post, gate))
        for V, step in _runs(T):
            for D in (ON_CHIP + step, 32768 // SIZE[T] + step, MOST):
                if D > ON_CHIP:
                    wide.add(_named(T, (V, 512 if D * SIZE[T] > 32768 else 256)))
    assert held["resnorm_kernel"] == forward
    assert held["resnorm_wide_kernel"] == wide
    assert held["resnorm_backward_kernel"] == back
    assert held["resnorm_staged_kernel"] == staged


def test_gated_projections(held):
    # the scale is fp16's; rows of whole runs are copied in fp32 alone
    assert held["gated_bound_kernel"] == {("__half", "0"), ("__half", "1")}
    assert held["gated_pad_kernel"] == {(T, str(read)) for T in RUN for read in
                                        ((0, 1, 2) if T == "float" else (0, 2))}
