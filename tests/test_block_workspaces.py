"""Where the product with an epilogue splits its sum it needs a workspace, and only there (host)."""
import pytest

from memory_bound_elementwise_amd.moe_block import linear_act_workspace, load_library

A = 1 << 20


def _call(m, n, k, ws, size):
    at = [A + (i << 40) for i in range(6)]
    return load_library().block_linear_act(at[0], at[1], None, None, at[4], m, n, k, 0, 0, ws and at[5] + ws - 1, size, None)


@pytest.mark.parametrize("m,n,k", [(33, 8, 2048), (100, 64, 7168), (40, 1024, 7168), (64, 64, 1 << 20)])
def test_split_sums(m, n, k):
    need = linear_act_workspace(m, n, k)
    assert need > 0 and need % (2 * m * n * 4) == 0      # an even number of partial products
    assert _call(m, n, k, None, 0) == 1 and _call(m, n, k, 1, need - 1) == 1
    assert _call(m, n, k, 5, need) == 2                    # not at 16 bytes


@pytest.mark.parametrize("m,n,k", [(0, 64, 7168), (8, 64, 1 << 16), (32, 4096, 7168), (33, 64, 512), (4096, 4096, 4096)])
def test_whole_sums(m, n, k):
    assert linear_act_workspace(m, n, k) == 0
