"""Workspace of the orthogonalised update: what its products keep between launches, and no more (host only)."""
import ctypes

import pytest

import sparse_moe_layer_biased_b200 as moe
from test_train_ops_host import FAKE, orth


@pytest.mark.parametrize("rows,cols", [(128, 2048), (2048, 128), (1, 1), (128, 128), (77, 2000), (1100, 17)])
def test_matrices_of_one_launch_need_no_workspace(rows, cols):
    """Shorter side up to 128, longer one up to 2048: all of it is on chip."""
    assert {moe.moe_orthogonalize_workspace_size(orth(n=n, rows=rows, cols=cols)) for n in (0, 1, 150, 65535)} == {256}
    d = orth(n=150, rows=rows, cols=cols)
    assert moe.lib().moe_orthogonalize(ctypes.byref(d), FAKE, None, FAKE, FAKE, 255, None) == 3
    assert moe.lib().moe_orthogonalize(ctypes.byref(d), FAKE, None, FAKE, None, 256, None) == 1


@pytest.mark.parametrize("rows,cols", [(129, 129), (128, 2049), (2049, 1), (200, 600), (4096, 1280)])
def test_matrices_of_several_launches(rows, cols):
    """Three arrays of X and three of A in 16 bits, rows padded to 64 elements: 6 bytes per padded element."""
    p = min(rows, cols)
    pad = lambda v: (v + 63) // 64 * 64  # noqa: E731
    for n in (1, 3):
        each = 6 * rows * pad(cols) + 6 * p * pad(p)
        size = moe.moe_orthogonalize_workspace_size(orth(n=n, rows=rows, cols=cols))
        # beside them the diagonals' remainders, the norms' parts and alignment
        assert n * each < size <= n * (each + 8 * pad(p) + 8 * 512) + 9 * 256
