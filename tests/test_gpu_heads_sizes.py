"""Ordinary heads at the ends of their ranges: many sequences, offsets beyond 32 bits, expanded heads, nothing to do."""
import pytest
import torch

from heads_util import check_sequence, normal
from test_gpu_heads_prep import check as check_prep, inputs
import test_gpu_heads_paged as paged
import test_gpu_heads_prompt as prompt

pytestmark = pytest.mark.gpu


def lengths(B, most, seed):
    return torch.randint(0, most + 1, (B,), generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.parametrize("paged_keys", [False, True])
@pytest.mark.parametrize("B", [32, 33, 257, 600])
def test_prompts_of_many_sequences(B, paged_keys):
    """Descriptions kept in lanes and searched for; the longest first and in order; the plan in one and two rounds."""
    lens = lengths(B, 40, B)
    lens[B // 2] = 700
    kw = dict(ctx=lengths(B, 100, 1), paged=True) if paged_keys else {}
    m = prompt.make(lens, H=2, Hkv=1, D=64, Dv=64, **kw)
    prompt.check(m, *prompt.run(m))


@pytest.mark.parametrize("B", [31, 33, 513, 1100])
def test_new_tokens_of_many_sequences(B):
    act = lengths(B, 200, B)
    act[0], act[-1] = 0, 9000
    m = paged.make(act, H=4, Hkv=2, D=64, Dv=64)
    paged.check(m, *paged.run(m))


def test_rows_beyond_32_bits():
    """Queries and outputs of more than 2^31 values: the first and the last sequences."""
    import mla_sparse_top_gb300 as mla
    H, D, n, B = 128, 128, 200, 670
    T = n * B
    assert T * H * D > 2 ** 31
    gen = torch.Generator().manual_seed(0)
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    k, v = normal(gen, (T, 1, D), q.dtype), normal(gen, (T, 1, D), q.dtype)
    for b in (0, B - 1):
        q[b * n:(b + 1) * n] = normal(gen, (n, H, D), q.dtype)
    cu = (torch.arange(B + 1, dtype=torch.int32) * n).cuda()
    out, lse = torch.empty((T, H, D), dtype=q.dtype, device="cuda"), torch.empty((T, H), device="cuda")
    dims = mla.prompt_dims(q, k, v, cu)
    ws = torch.empty(mla.mla_prompt_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mla.mla_prompt_attn_fwd(q, k, v, cu, out, lse, ws, softmax_scale=0.1, dims=dims)
    assert mla.heads_device_status(clear=True) == 0
    for b in (0, B - 1):
        r = slice(b * n, (b + 1) * n)
        check_sequence(out[r], lse[r], q[r], k[r], v[r], 0.1, True, f"sequence {b}")


def test_far_pages_of_a_prompt_and_of_appended_rows():
    """Pages whose offset passes 2^31 values: written by the append, read by the prompt's chunk."""
    import mla_sparse_top_gb300 as mla
    blocks, Hkv, D, n = 80000, 2, 128, 200
    pool = torch.empty((blocks, 128, 2, Hkv, D), dtype=torch.bfloat16, device="cuda")  # keys and values share pages
    kc, vc = pool[:, :, 0], pool[:, :, 1]
    k, pos = inputs(n, Hkv, D, torch.bfloat16, seed=1)
    v, _ = inputs(n, Hkv, D, torch.bfloat16, seed=2)
    pages = torch.tensor([blocks - 1, blocks - 3])
    rows = torch.cat([pages[0] * 128 + torch.arange(128), pages[1] * 128 + torch.arange(n - 128)]).cuda()
    mla.mla_kv_append(pos, rows, k, v, kc, vc, params=mla.rope_params(), rot_dim=64)
    flat_k, flat_v = torch.cat([kc[pages[0]], kc[pages[1]]])[:n], torch.cat([vc[pages[0]], vc[pages[1]]])[:n]
    check_prep(flat_k, k, pos, None, {}, "keys", rot_dim=64, rot_off=0, half=False)
    assert torch.equal(flat_v, v)
    q, _ = inputs(90, 4, D, torch.bfloat16, seed=3)
    cu, act = torch.tensor([0, 90], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    table = pages.to(torch.int32)[None].cuda()
    out, lse = torch.empty_like(q), torch.empty((90, 4), device="cuda")
    dims = mla.prompt_dims(q, kc, vc, cu, block_table=table)
    ws = torch.empty(mla.mla_prompt_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mla.mla_prompt_attn_fwd(q, kc, vc, cu, out, lse, ws, block_table=table, act_seqs=act, softmax_scale=0.02, dims=dims)
    assert mla.heads_device_status(clear=True) == 0
    check_sequence(out, lse, q, flat_k.cpu(), flat_v.cpu(), 0.02, True, "far pages")


def test_expanded_heads():
    """One key and value head in memory, seen as four (a head stride of 0); queries of one token for all."""
    import mla_sparse_top_gb300 as mla
    gen = torch.Generator().manual_seed(3)
    n, H, Hkv, D = 150, 8, 4, 64
    k1, v1 = normal(gen, (n, 1, D), torch.bfloat16), normal(gen, (n, 1, D), torch.bfloat16)
    q = normal(gen, (n, H, D), torch.bfloat16)
    k, v = k1.expand(n, Hkv, D), v1.expand(n, Hkv, D)
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    out, lse = torch.empty_like(q), torch.empty((n, H), device="cuda")
    dims = mla.prompt_dims(q, k, v, cu)
    ws = torch.empty(mla.mla_prompt_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    mla.mla_prompt_attn_fwd(q, k, v, cu, out, lse, ws, softmax_scale=0.125, dims=dims)
    assert mla.heads_device_status(clear=True) == 0
    check_sequence(out, lse, q, k.contiguous(), v.contiguous(), 0.125, True, "expanded")
    y = torch.empty((n, Hkv, D), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    mla.mla_norm_rope(pos, k, params=mla.rope_params(), rot_dim=64, out=y)
    check_prep(y, k, pos, None, {}, "expanded", rot_dim=64, rot_off=0, half=False)


def test_nothing_to_do():
    """No tokens and no sequences: no launch, nothing written."""
    import mla_sparse_top_gb300 as mla
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = torch.full((3, 128, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    other = pool.clone()
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    mla.mla_norm_rope(torch.empty(0, **i32), none, params=mla.rope_params(), rot_dim=64)
    mla.mla_kv_append(torch.empty(0, **i32), torch.empty(0, dtype=torch.int64, device="cuda"), none, none, pool, other,
                      params=mla.rope_params(), rot_dim=64)
    lse, ws = torch.empty((0, 2), device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda")
    mla.mla_paged_attn_fwd(none, pool, other, torch.zeros((0, 4), **i32), torch.empty(0, **i32), none.clone(), lse, ws,
                           softmax_scale=1.0)
    mla.mla_prompt_attn_fwd(none, none, none, torch.zeros(1, **i32), none.clone(), lse, ws, softmax_scale=1.0)
    mla.mla_prompt_attn_fwd(none, none, none, torch.zeros(3, **i32), none.clone(), lse, ws, softmax_scale=1.0)
    # rows, and no sequence that has one
    q = torch.ones((7, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, l7 = torch.full_like(q, 3.0), torch.full((7, 2), 3.0, device="cuda")
    mla.mla_prompt_attn_fwd(q, q.clone(), q.clone(), torch.tensor([4, 4, 4], **i32), out, l7, ws, softmax_scale=1.0)
    assert mla.heads_device_status(clear=True) == 0
    assert (pool == 5).all() and (out == 3).all() and (l7 == 3).all()


def test_offsets_that_run_back_and_forth():
    """Sequences that would be far more than the rows there are: reported, nothing out of place is touched."""
    import mla_sparse_top_gb300 as mla
    T, H, D = 64, 2, 64
    gen = torch.Generator().manual_seed(5)
    q, k, v = (normal(gen, (T, H, D), torch.bfloat16) for _ in range(3))
    cu = torch.tensor([0, T] * 500 + [0], dtype=torch.int32).cuda()  # every second one has all rows
    guard = torch.full((T + 512, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    out, lse = guard[256:256 + T], torch.empty((T, H), device="cuda")
    dims = mla.prompt_dims(q, k, v, cu)
    ws = torch.empty(max(256, mla.mla_prompt_workspace_bytes(dims)), dtype=torch.uint8, device="cuda")
    mla.mla_prompt_attn_fwd(q, k, v, cu, out, lse, ws, softmax_scale=0.125, dims=dims)
    assert mla.heads_device_status(clear=True) == mla.MLA_DEVICE_BAD_LENGTH
    assert (guard[:256] == 3).all() and (guard[256 + T:] == 3).all()
    check_sequence(out, lse, q, k, v, 0.125, True, "the rows that each of them has")
