"""The residual norm's gradient where values are not finite, and over many rows that start anywhere."""
import pytest
import torch

from test_gpu_residual_norm import TYPES, _check, _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("which", ["dS", "dY", "S", "Z", "Stats"])
@pytest.mark.parametrize("rows,groups,D", [(60, 6, 48), (60, 60, 77), (900, 300, 600), (60, 0, 1031),
                                           (40, 4, 6000), (12, 3, 9001)])
def test_rows_that_are_not_finite_stay_by_themselves(gs_cuda, rows, groups, D, which, value, dtype):
    """The other rows of dX and dZ, and the other gates' gradients, keep their bits; sums over all rows
    are NaN where the row has a share in them."""
    t, dS, dY = _make(rows, D, dtype, True, groups, seed=D)
    S, _, stats = gs_cuda.gs_residual_norm(**t)
    form = {k: t[k] for k in ("gate", "z_scale", "z_B")}
    given = dict(dS=dS, dY=dY, S=S, Z=t["Z"], Stats=stats)
    want = gs_cuda.gs_residual_norm_backward(**given, Scale=t["Scale"], bias=True, **form)
    row = 7
    # the third column, or the deviation of S
    given[which][row, 3 if which == "Stats" else 2] = value
    got = gs_cuda.gs_residual_norm_backward(**given, Scale=t["Scale"], bias=True, **form)
    for k in ("dX", "dZ", "dgate"):
        if k not in got:
            continue
        at = row * groups // rows if k == "dgate" else row
        others = torch.arange(got[k].shape[0], device="cuda") != at
        assert torch.equal(got[k][others], want[k][others]), k
    assert not torch.isfinite(got["dZ"][row]).all()
    if which == "dY":
        assert torch.equal(torch.isfinite(got["dB"]), torch.arange(D, device="cuda") != 2)
    assert gs_cuda.gs_device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,D,groups", [(4000, 771, 1), (4000, 771, 40), (9000, 300, 0)])
def test_many_rows_that_start_anywhere(gs_cuda, rows, D, groups, dtype):
    """Tensors that start and end between 16-byte boundaries, with more rows than are on their way at
    once: the places of the outermost rows, which are not copied whole, are used again."""
    t, dS, dY = _make(rows, D, dtype, True, groups, seed=4)

    def moved(x):
        room = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)
        room[1:] = x.flatten()
        return room[1:].view(x.shape)

    t = {k: None if v is None else moved(v) for k, v in t.items()}
    dS, dY = moved(dS), moved(dY)
    S, _, stats, _ = _check(gs_cuda, t, dS, dY, dtype)
    form = {k: t[k] for k in ("gate", "z_scale", "z_B")}
    S = moved(S)
    back = [gs_cuda.gs_residual_norm_backward(dS, dY, S, t["Z"], stats, t["Scale"], bias=True, **form)
            for _ in range(3)]
    for one in back[1:]:
        for k in one:
            assert torch.equal(one[k], back[0][k]), k
