"""The calls around a drafted decode step at the ends of their integer ranges, on the host."""
import ctypes

import pytest

from test_step_abi_host import lib  # noqa: F401

MANY = 1 << 20


def workspace(lib, **kw):  # noqa: F811
    from mla_sparse_top_gb300.binding import MlaDims
    d = dict(B=1, S1=1, n_q=128, n_kv=1, d_nope=512, d_rope=64, block_size=128, num_blocks=16, max_blocks_per_seq=100,
             topk=0, kv_dtype=0)
    return lib.mla_tree_workspace_bytes(ctypes.byref(MlaDims(**{**d, **kw})))


@pytest.mark.parametrize("B", [1, 2, 3, 4, 8, 12, 15])
@pytest.mark.parametrize("S1,n_q", [(MANY, 128), (MANY, 1), (MANY // 2, 64), (64, 128)])
@pytest.mark.parametrize("W", [1 << 23, (1 << 23) - 1, 1 << 20])
def test_tree_workspace_of_the_largest_dims(lib, B, S1, n_q, W):  # noqa: F811
    """As much as any call with a team for every cluster needs, never less."""
    full = workspace(lib, B=64, S1=8, max_blocks_per_seq=1000)
    assert full > 76 * 4 * 128 * 256 * 4
    assert workspace(lib, B=B, S1=S1, n_q=n_q, max_blocks_per_seq=W) == full


def test_tree_workspace_grows_up_to_that(lib):  # noqa: F811
    sizes = [workspace(lib, B=B, max_blocks_per_seq=W) for B, W in ((1, 1), (1, 4), (2, 4), (8, 8), (64, 64), (4096, 512))]
    assert sizes == sorted(sizes) and sizes[0] < sizes[3] < sizes[4] == sizes[5]
