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
