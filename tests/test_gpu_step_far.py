"""The calls around a drafted decode step at their far ends: offsets beyond 32
bits, drafts of thousands of tokens, many sequences.  What a far row gives must
be, bit for bit, what the same row gives in a small call."""
import numpy as np
import pytest
import torch

from oracle import step
from test_gpu_tree import HALF, U, check, make

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("dtype,H,D", [(BF16, 128, 192), (torch.float32, 67, 131)])  # 16-byte rows, single values
def test_rotation_of_more_than_2_to_32_bytes_and_values(dtype, H, D):
    import mla_sparse_top_gb300 as mla
    T = (1 << 32) // (H * D) + 1000
    x = torch.empty((T, H, D), dtype=dtype, device="cuda")
    x.view(-1, D)[::7] = 1.5  # a few values; the rows compared get random ones
    at = [0, T // 2, T - 1, (1 << 31) // (H * D), (1 << 31) // (H * D * x.element_size()), (1 << 32) // (H * D)]
    x[at] = torch.randn((len(at), H, D), device="cuda").to(dtype)
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 37
    kw = dict(params=mla.rope_params(), rot_dim=64, rot_off=64, half=dtype != BF16)
    rows = x[at].clone()
    want = torch.empty_like(rows)
    mla.mla_rope_apply(pos[at].contiguous(), rows, out=want, **kw)
    mla.mla_rope_apply(pos, x, **kw)
    assert torch.equal(x[at], want)


def test_keys_to_rows_beyond_2_to_32_values():
    import mla_sparse_top_gb300 as mla
    rows = (1 << 32) // 128 + 500
    cache = torch.zeros((rows, 1, 128), dtype=BF16, device="cuda")
    k, q = torch.randn((4, 1, 128), device="cuda").to(BF16), torch.randn((4, 2, 128), device="cuda").to(BF16)
    where = torch.tensor([rows - 1, 5, (1 << 24) + 3, rows], device="cuda")
    pos = torch.tensor([9, 10, 11, 12], dtype=torch.int32, device="cuda")
    want = torch.empty_like(k)
    kw = dict(params=mla.rope_params(), rot_dim=64)
    mla.mla_rope_apply(pos, q.clone(), k, k_out=want, **kw)
    mla.mla_rope_apply(pos, q, k, k_out=cache, k_rows=where, **kw)
    assert torch.equal(cache[where[:3]], want[:3])
    assert mla.rope_device_status(clear=True) == mla.MLA_DEVICE_BAD_BLOCK  # the last one lies behind the cache


def test_page_plan_with_the_largest_block_ids():
    import mla_sparse_top_gb300 as mla
    n = (1 << 24) - 1
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = t([[n - 1, -1, -1], [3, -1, -1]])
    act, slots = t([0, 0]), torch.zeros(8, dtype=torch.int64, device="cuda")
    mla.mla_page_plan(t([126, 128]), None, t([n - 2, n - 3, 7]), table, act, slots, S1=4, num_blocks=n)
    first, second, third = (n - 1) * 128, (n - 2) * 128, (n - 3) * 128
    assert slots.tolist() == [first + 126, first + 127, second, second + 1, third, third + 1, third + 2, third + 3]
    assert mla.page_device_status(clear=True) == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("tree", [False, True])
def test_drafts_of_thousands_of_tokens(tree, int8):
    """A prompt as one chain, or a tree of as many tokens: mask rows of 33 words, 33 row blocks."""
    assert check(make(70, [2300, 2100], 2101, 2, int8=int8, tree=tree, lens=[2101, 1900])) == 0


def test_more_sequences_than_a_grid_dimension():
    """70,000 sequences of one to three positions; three row blocks a sequence for the INT8 expansion's grid."""
    import mla_sparse_top_gb300 as mla
    B, S1, n_q = 70_000, 3, 100
    g = torch.Generator(device="cuda").manual_seed(1)
    act = torch.randint(1, 4, (B,), generator=g, device="cuda", dtype=torch.int32)
    pool = 512  # pages, shared by the sequences
    table = torch.randint(0, pool, (B, 1), generator=g, device="cuda", dtype=torch.int32)
    kv = torch.randint(-127, 128, (pool * 128, 512), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    sc = (torch.rand((pool * 128, 4), generator=g, device="cuda") + 0.5) / 64
    kr = torch.randn((pool * 128, 64), generator=g, device="cuda").to(BF16)
    qn = torch.randn((B * S1, n_q, 512), generator=g, device="cuda", dtype=BF16)
    qr = torch.randn((B * S1, n_q, 64), generator=g, device="cuda", dtype=BF16)
    out = torch.empty_like(qn)
    dims = mla.tree_dims(qn, kv, table, S1=S1)
    ws = torch.empty(mla.mla_tree_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mla.mla_tree_attn_fwd(qn, qr, kv, kr, sc, table, act, out, None, ws, dims=dims)
    assert mla.tree_device_status(clear=True) == 0
    lat = (kv.float() * sc.repeat_interleave(128, 1)).to(BF16).double().cpu().numpy()
    rope = kr.double().cpu().numpy()
    top = float(np.linalg.norm(np.concatenate([lat, rope], 1), axis=1).max()
                * torch.cat([qn, qr], -1).float().norm(dim=-1).max())
    for b in (0, 1, 33_333, 65_534, 65_535, 65_536, B - 1):
        rows = slice(b * S1, b * S1 + S1)
        o, _, mag = step.tree_attention(qn[rows].double().cpu().numpy(), qr[rows].double().cpu().numpy(), lat, rope,
                                        table[b:b + 1].cpu().numpy(), act[b:b + 1].cpu().numpy(), None, None, S1, 576 ** -0.5)
        d = 576 ** -0.5 * top * 578 * U + 19 * U  # the bound of test_gpu_tree.py, for three keys
        bound = (HALF + 2 * d) * mag * (1 + 2 * d) + HALF * np.abs(o) * 1.01 + 1e-30
        assert (np.abs(out[rows].double().cpu().numpy() - o) <= bound).all(), b
