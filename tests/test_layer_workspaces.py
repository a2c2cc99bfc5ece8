"""Sizes of the scratch memory that the layer operators ask for (no GPU needed)."""
import pytest

import nvfp4_bit_block_gb300 as nv


@pytest.fixture(scope="module")
def L():
    nv.build()
    return nv.layer_lib()


@pytest.mark.parametrize("N", [1, 133, 5120, 20480, 33001])
@pytest.mark.parametrize("M", [1, 2, 7, 100, 607])
def test_the_norm_gradients_workspace_follows_the_rows(L, M, N):
    """Few rows leave few rows of partial sums: at most one for each, and two sums per row."""
    n = L.nvfp4_layernorm_backward_workspace(M, N)
    assert 0 <= n <= M * 2 * N * 4 + (M + 1) * 8


def test_the_norm_gradients_workspace_of_many_rows_stays_bounded(L):
    assert L.nvfp4_layernorm_backward_workspace(16384, 5120) <= 30e6
