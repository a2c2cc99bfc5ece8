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


@pytest.mark.parametrize("M,N", [(1, 1), (257, 33), (16384, 20480), (16384, 131072), (1000000, 64), (2 ** 31 - 1, 8),
                                 (2 ** 31 - 1, 9)])
def test_the_epilogue_gradients_workspace_stays_within_a_grid(L, M, N):
    """Partial sums of at most 65535 bands (the most blocks of a grid's second dimension)."""
    n = L.nvfp4_act_backward_workspace(M, N)
    assert 0 <= n <= 65535 * N * 4


@pytest.mark.parametrize("M", [608, 5000, 16384, 10 ** 6, 2 ** 31 - 1])
def test_the_norm_gradients_workspace_grows_with_a_part_for_every_510_rows(L, M):
    n = L.nvfp4_layernorm_backward_workspace(M, 64)
    assert 0 <= n <= (608 + 2 + M / 510) * 2 * 64 * 4 + (M + 1) * 8
