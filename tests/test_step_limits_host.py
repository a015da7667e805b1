"""The calls around a drafted decode step at the ends of their integer ranges, on the host."""
import ctypes

import pytest
import torch

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


class Shaped:
    """As much of a tensor as the binding looks at, of any size."""

    def __init__(self, dtype, *shape, stride=None):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), "cuda:0"
        self._stride = stride or tuple(torch.Size(shape[i + 1:]).numel() for i in range(len(shape)))

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return self._stride

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0  # a call that went on would be refused for its null pointers


I32, I64, F32, BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16


@pytest.fixture
def mla(monkeypatch, lib):  # noqa: F811
    import mla_sparse_top_gb300 as mla
    from mla_sparse_top_gb300 import binding
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda stream, dev: 0)
    return mla


@pytest.mark.parametrize("over", [1 << 31, (1 << 32) + 8, (1 << 33) + 6])
def test_binding_refuses_sizes_beyond_32_bits(mla, over):
    def plan(B=2, S1=0, T=8, W=4, F=5, num_blocks=9):
        mla.mla_page_plan(Shaped(I32, B), Shaped(I32, B), Shaped(I32, F), Shaped(I32, B, W), Shaped(I32, B),
                          Shaped(I64, T), S1=S1, num_blocks=num_blocks)
    for kw in (dict(B=over), dict(S1=over), dict(T=over), dict(W=over), dict(F=over), dict(num_blocks=over)):
        with pytest.raises(ValueError, match="32 bits"):
            plan(**kw)
    params = mla.rope_params()
    with pytest.raises(ValueError, match="32 bits"):
        mla.mla_rope_table(Shaped(I32, over), Shaped(F32, over, 32), Shaped(F32, over, 32), params=params)

    def rotate(T=4, H=2, D=64, rot_dim=64, rot_off=0):
        mla.mla_rope_apply(Shaped(I32, T), Shaped(BF16, T, H, D), params=params, rot_dim=rot_dim, rot_off=rot_off)
    for kw in (dict(T=over), dict(H=over), dict(D=over), dict(rot_dim=over), dict(rot_off=over)):
        with pytest.raises(ValueError, match="32 bits"):
            rotate(**kw)
    for q, kv, table in (((over, 1, 512), 128, (over, 1)), ((1, over, 512), 128, (1, 1)), ((1, 1, 512), 128 * over, (1, 1)),
                         ((1, 1, 512), 128, (1, over))):
        with pytest.raises(ValueError, match="32 bits"):
            mla.tree_dims(Shaped(BF16, *q), Shaped(BF16, kv, 512), Shaped(I32, *table), S1=1)


def test_binding_leaves_smaller_sizes_to_the_library(mla):
    for S1 in (-1, -(1 << 31)):
        with pytest.raises(mla.MlaError) as e:
            mla.mla_page_plan(Shaped(I32, 2), Shaped(I32, 2), Shaped(I32, 5), Shaped(I32, 2, 4), Shaped(I32, 2),
                              Shaped(I64, 8), S1=S1, num_blocks=9)
        assert e.value.status == -2
