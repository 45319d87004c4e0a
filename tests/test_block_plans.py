"""What the binding of the transformer-block operators keeps from one call for the next: shapes
and numbers, never an object whose value may change."""
import pytest
import torch

import spatial_transformer_sampling_gb300 as gs
from spatial_transformer_sampling_gb300 import block


def _plan_of(**kw):
    """The plan of a call on CPU tensors, which the binding refuses only after it has it."""
    block._PLANS.clear()
    t = torch.zeros((2, 6, 3, 8))
    with pytest.raises(ValueError, match="CUDA"):
        gs.gs_attention(t, t, t, **kw)
    (plan,) = block._PLANS.values()
    return plan


def test_scale_given_as_a_tensor_is_read_at_every_call():
    scale = torch.tensor(0.5)
    assert _plan_of(scale=scale).attrs.scale == 0.5
    t = torch.zeros((2, 6, 3, 8))
    scale.fill_(2.0)
    with pytest.raises(ValueError, match="CUDA"):
        gs.gs_attention(t, t, t, scale=scale)
    assert sorted(p.attrs.scale for p in block._PLANS.values()) == [0.5, 2.0]
    for key in block._PLANS:
        assert not any(isinstance(part, torch.Tensor) for part in key)


def test_axis_given_as_a_tensor_is_read_at_every_call():
    t, axis = torch.zeros((2, 6)), torch.tensor(0)
    for value in (0, 1):
        axis.fill_(value)
        with pytest.raises(ValueError, match="CUDA"):
            gs.gs_layer_norm(t, torch.ones(6), axis=axis)
    before = block._norm_dims.cache_info().currsize
    axis.fill_(2)
    with pytest.raises(ValueError, match="out of range"):
        gs.gs_layer_norm(t, torch.ones(6), axis=axis)
    assert block._norm_dims.cache_info().currsize == before


def test_heads_of_width_zero_are_refused():
    t = torch.zeros((2, 6, 3, 0))
    with pytest.raises(ValueError, match="width 0"):
        gs.gs_attention(t, t, t)


@pytest.mark.gpu
def test_results_follow_a_scale_that_changes_in_place(gs_cuda):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    Q, K, V, dO = (torch.randn((2, 40, 2, 32), generator=g, device="cuda") for _ in range(4))
    scale = torch.tensor(0.5)
    first = gs_cuda.gs_attention(Q, K, V, scale=scale)
    gs_cuda.gs_attention_backward(dO, Q, K, V, *first, scale=scale)
    scale.fill_(0.125)
    got = gs_cuda.gs_attention(Q, K, V, scale=scale)
    want = gs_cuda.gs_attention(Q, K, V, scale=0.125)
    assert not torch.equal(first[0], want[0])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for a, b in zip(gs_cuda.gs_attention_backward(dO, Q, K, V, *want, scale=scale),
                    gs_cuda.gs_attention_backward(dO, Q, K, V, *want, scale=0.125)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("q,k", [([2, 3], None), (None, [3, 2]), ([2, 3], (3, 2)), (None, None),
                                 (torch.Size((2, 3)), [1, 6])])
def test_extents_in_any_sequence_or_left_out(q, k):
    at = _plan_of(q_extent=q, k_extent=k).attrs
    assert tuple(at.q_extent) == tuple(q or (1, 6)) and tuple(at.k_extent) == tuple(k or (1, 6))


@pytest.mark.parametrize("q", [(), (6,), (1, 2, 3), (2, 2)])
def test_extents_of_another_shape_are_refused(q):
    t = torch.zeros((2, 6, 3, 8))
    with pytest.raises(ValueError, match="extent"):
        gs.gs_attention(t, t, t, q_extent=q)
