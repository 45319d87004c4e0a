"""Attention between two unequal grids of tokens on the GPU, against the 64-bit reference."""
import pytest

from test_gpu_attention import DTYPES, Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("q", [(1, 226), (1, 240)])
def test_bias_gradient_where_a_step_crosses_one_row_more_than_its_keys(gs_cuda, q, dtype):
    # keys in rows of 63: from the last of a row on, the 64th key after it lies two rows below;
    # a bias entry per offset shows a sum that lands in another's place
    Problem(gs_cuda, 500, dtype, 1, 1, 16, q, (70, 63), 0).both()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("D", [96, 128])
@pytest.mark.parametrize("q,k", [((20, 8), (4, 130)), ((16, 8), (3, 128)), ((40, 16), (40, 208)),
                                 ((1, 32), (32, 1)), ((8, 8), (1, 224)), ((16, 16), (1, 256)),
                                 ((32, 8), (32, 128))])
def test_gradient_of_wide_heads_between_narrow_and_wide_grids(gs_cuda, q, k, D, dtype):
    # the windows of the bias and of its gradient together are more than a block's shared memory
    Problem(gs_cuda, 510, dtype, 1, 2, D, q, k, 8).both()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("q,k", [((9, 16), (13, 40)), ((13, 40), (9, 16)), ((3, 7), (11, 29)),
                                 ((1, 90), (12, 12)), ((12, 12), (1, 90))])
def test_unequal_grids(gs_cuda, q, k, dtype):
    Problem(gs_cuda, 520, dtype, 2, 2, 80, q, k, 0, k_len=[k[0] * k[1], k[0] * k[1] // 2 + 3]).both()
