"""Sequences of 2^27 keys and more of which only a few pages exist: the others are masked out and reported."""
import numpy as np
import pytest
import torch

from heads_util import cache, check_sequence, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length,Dv,S1,H", [((1 << 27) + 600, 128, 1, 8), ((1 << 28) + 600, 64, 3, 8), (1 << 30, 128, 1, 4),
                                            ((1 << 27) + 1, 128, 2, 40)])
def test_few_pages_of_a_long_sequence(length, Dv, S1, H):
    import mla_sparse_top_gb300 as mla
    gen = torch.Generator().manual_seed(S1)
    D, blocks, W = 64, 5, -(-length // 128)
    k, v = cache(blocks, 1, D, "token", torch.bfloat16, gen=gen), cache(blocks, 1, Dv, "token", torch.bfloat16, gen=gen)
    q = normal(gen, (S1, H, D), torch.bfloat16)
    table = torch.full((1, W), -1, dtype=torch.int32)
    pages = {5: 3, W // 2: 0, W - 1: 4}  # place in the table: page
    for at, page in pages.items():
        table[0, at] = page
    table[0, 7] = blocks  # one behind the pool's last
    table, act = table.cuda(), torch.tensor([length], dtype=torch.int32).cuda()
    out, lse = torch.empty((S1, H, Dv), dtype=q.dtype, device="cuda"), torch.empty((S1, H), device="cuda")
    dims = mla.paged_dims(q, k, v, table, S1=S1)
    ws = torch.empty(mla.mla_paged_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mla.mla_paged_attn_fwd(q, k, v, table, act, out, lse, ws, softmax_scale=0.125, S1=S1, dims=dims)
    assert mla.heads_device_status(clear=True) == mla.MLA_DEVICE_BAD_BLOCK
    # their keys one behind the other: the tokens are the newest of these too
    rows = [(page, min(128, length - 128 * at)) for at, page in pages.items()]
    keys, values = (torch.cat([x.cpu()[page, :n] for page, n in rows]) for x in (k, v))
    check_sequence(out, lse, q, keys, values, 0.125, True, "three pages", np.ones(len(keys), bool))
