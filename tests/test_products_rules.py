"""Which kernel takes a product by expert, as far as the host shows it: streamed
calls need no workspace, fp32 calls in tiles do."""
import pytest

import swiglu_mlp_top_gb300 as mm  # noqa: F401
from swiglu_mlp_top_gb300 import _lib as L


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return L.load()


@pytest.mark.parametrize("E", [1, 8, 64])
def test_few_fp32_rows_are_streamed(lib, E):
    """Up to 32 rows an expert and 32 more: all of them on one expert take at
    most about twice the tiles' time."""
    need = lambda rows, K: lib.mm_grouped_matmul_workspace_bytes(rows, K, 1024, E, L.MM_DTYPE_F32)  # noqa: E731
    assert need(32 + 32 * E, 2048) == 0 and need(32 + 32 * E + 1, 2048) > 0
    # rows that do not start on 16 bytes: multiply-adds up to 4 rows an expert and 16 more
    assert need(16 + 4 * E, 2049) == 0 and need(16 + 4 * E + 1, 2049) > 0


def test_fp32_gradients_always_have_scratch(lib):
    assert lib.mm_grouped_matmul_backward_workspace_bytes(1, 64, 64, 4, L.MM_DTYPE_F32) > 256
