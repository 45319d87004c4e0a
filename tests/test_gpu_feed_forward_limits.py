"""The feed-forward operators beyond 2^31 elements, and errors that stay with their call."""
import pytest
import torch

import feed_forward_reference as ref
from test_gpu_block_errors import _BrokenCapture

pytestmark = pytest.mark.gpu


def _rows_of(n):
    """A few rows at the start, around 2^31 elements of 4096 and 2048, and at the end."""
    return torch.tensor([0, 1, 255, 256, (1 << 31) // 4096 - 1, (1 << 31) // 4096, n - 257, n - 1])


def test_gated_linear_beyond_32_bit_offsets(gs_cuda):
    rows, D, F = 540001, 16, 4096   # 2.2e9 outputs
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    X, Wg, Wu, bg, bu = mk(rows, D), mk(F, D) * 0.25, mk(F, D) * 0.25, mk(F), mk(F)
    H, G, U = gs_cuda.gs_gated_linear(X, Wg, Wu, bg, bu, keep=True)
    at = _rows_of(rows).cuda()
    ref.check_gated((H[at], G[at], U[at]), X[at], Wg, Wu, bg, bu, "silu", "bfloat16")
    back = gs_cuda.gs_gated_linear_backward(H, X, Wg, Wu, G, U, bias=True)
    want, plain, floor = ref.gated_backward(H[at], X[at], Wg, Wu, G[at], U[at], "silu")
    ref.check(back[0][at], want[0], floor[0], "bfloat16", ref.terms(2 * F), plain[0] * 1.02, "dX")
    # the sums over all rows, a few of the outputs at a time
    for f in (slice(0, 3), slice(F - 3, F)):
        part = lambda t: t[:, f].contiguous()
        want, plain, floor = ref.gated_backward(part(H), X, Wg[f], Wu[f], part(G), part(U), "silu")
        for i in (1, 2, 3, 4):
            ref.check(back[i][f], want[i], floor[i], "bfloat16", ref.terms(rows),
                      plain[i] * 1.02 if i < 3 else 0.0, str(i))
    assert gs_cuda.gs_device_status() == 0


@pytest.mark.parametrize("D,rows", [(4096, 530000), (8200, 265000)])
def test_residual_norm_beyond_32_bit_offsets(gs_cuda, rows, D):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    X, Z, a, b, gate = mk(rows, D), mk(rows, D), mk(D), mk(D), mk(1, D)
    form = dict(gate=gate, z_scale=a, z_B=b)
    S, Y, st = gs_cuda.gs_residual_norm(X, Z, b, a, **form)
    at = _rows_of(rows)[[0, 2, 6, 7]].cuda()
    refs, sums = ref.residual_norm(X[at], Z[at], b, a, kind="layer", alpha=1.0, eps=1e-5, **form)
    C = ref.terms(D)
    for got, r, A, dt in zip((S, Y, st), refs, sums, ("bfloat16", "bfloat16", "float32")):
        ref.check(got[at], r, A, dt, C)
    back = gs_cuda.gs_residual_norm_backward(X, Y, S, Z, st, b, bias=True, **form)
    want = ref.residual_norm_backward(X[at], Y[at], S[at], Z[at], st[at], b, kind="layer", alpha=1.0,
                                      **form)
    for k in ("dX", "dZ"):
        ref.check(back[k][at], *want[k], "bfloat16", C, what=k)
    few = slice(D - 5, D)
    Yc, hat = Y[:, few].double().cpu(), ((S[:, few].double() - st[:, 2:3]) * st[:, 3:4]).cpu()
    ref.check(back["dB"][few], Yc.sum(0), Yc.abs().sum(0), "bfloat16", ref.terms(rows))
    ref.check(back["dScale"][few], (Yc * hat).sum(0), (Yc * hat).abs().sum(0) * 2, "bfloat16",
              ref.terms(rows))
    assert gs_cuda.gs_device_status() == 0


def test_an_error_stays_with_its_call(gs_cuda):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda")
    calls = {}
    for name, dt in ref.DT.items():
        for rows in (3, 200):
            X, W, b, dH = mk(rows, 65).to(dt), mk(40, 65).to(dt), mk(40).to(dt), mk(rows, 40).to(dt)
            H, G, U = gs_cuda.gs_gated_linear(X, W, W, b, b, keep=True)
            calls[f"gated {name} {rows}"] = lambda X=X, W=W, b=b: gs_cuda.gs_gated_linear(X, W, W, b, b)
            calls[f"gated back {name} {rows}"] = (
                lambda dH=dH, X=X, W=W, G=G, U=U: gs_cuda.gs_gated_linear_backward(dH, X, W, W, G, U,
                                                                                   bias=True))
        none = mk(0, 65).to(dt)
        calls[f"gated no row {name}"] = lambda n=none, W=W: gs_cuda.gs_gated_linear_backward(
            n[:, :40].contiguous(), n, W, W, n[:, :40].contiguous(), n[:, :40].contiguous())
        for D in (40, 600, 9000):
            X, a, gate = mk(6, D).to(dt), mk(D).to(dt), mk(2, D).to(dt)
            form = dict(gate=gate, z_scale=a, z_B=a)
            S, Y, st = gs_cuda.gs_residual_norm(X, X, a, a, **form)
            calls[f"norm {name} {D}"] = lambda X=X, a=a, f=form: gs_cuda.gs_residual_norm(X, X, a, a, **f)
            calls[f"norm back {name} {D}"] = (
                lambda X=X, S=S, st=st, a=a, f=form: gs_cuda.gs_residual_norm_backward(
                    X, X, S, X, st, a, bias=True, **f))
    X, a = mk(4, 8), mk(8)
    torch.cuda.synchronize()
    wrong = []
    for name, call in calls.items():
        with _BrokenCapture():
            try:
                call()
                wrong.append(f"{name}: no error on a stream that refuses it")
            except gs_cuda.GsError as e:
                assert e.status == 7, e
        try:
            gs_cuda.gs_layer_norm(X, a)
            gs_cuda.gs_gated_linear(X, X, X)
        except gs_cuda.GsError as e:
            wrong.append(f"{name} left an error: {e}")
    torch.cuda.synchronize()
    assert not wrong, wrong
    assert gs_cuda.gs_device_status() == 0
