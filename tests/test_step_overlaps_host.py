"""Outputs that overlap inputs or one another are refused before any CUDA call
(fake addresses; every call below is refused).  Skipped where there is a GPU: a
call that was not refused would go to those addresses."""
import ctypes

import pytest
import torch

from test_step_abi_host import lib, page_args, ptr, rope_call, rope_params, tree_call  # noqa: F401

UNSUPPORTED = -4
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses stay off a GPU")


# q: 8 tokens x 4 heads x 192 bf16 values from ptr(0) to ptr(1), 12288 bytes each
@pytest.mark.parametrize("tensor", [
    dict(out=ptr(0) + 2), dict(out=ptr(0) + 128 * 2), dict(out=ptr(0) + 12286), dict(x=ptr(1) + 12286),
    dict(out=ptr(0) + 192 * 2),                                           # a head further on
    dict(out=ptr(0) + 4 * 192 * 2),                                       # a token further on
    dict(x=ptr(1) + 64, x_token_stride=0, x_head_stride=0),               # a broadcast input inside the output
    dict(out=ptr(0) + 100, out_token_stride=5 * 192, out_head_stride=240),  # other strides
    dict(out=ptr(9) - 12288 + 16),                                        # positions in the last token
    dict(out=ptr(9) + 28),                                                # the last position
    dict(rows=ptr(1) + 64, num_rows=8),                                   # the list of rows in the output
    dict(x=ptr(60), rows=ptr(5), num_rows=100, out=ptr(60) - 1536 * 99),   # the cache's last row is the first token
])
def test_rope_apply_refuses_overlaps(lib, tensor):  # noqa: F811
    assert rope_call(lib, None, tensor) == UNSUPPORTED
    assert lib.mla_rope_last_error()
    apart = dict(x=ptr(100), out=ptr(101))
    assert rope_call(lib, None, apart, tensor) == UNSUPPORTED


@pytest.mark.parametrize("k", [
    dict(x=ptr(50), out=ptr(1)), dict(x=ptr(50), out=ptr(1) + 12286), dict(x=ptr(1) + 12286, out=ptr(50)),
    dict(x=ptr(50), out=ptr(0) + 1536), dict(x=ptr(0), out=ptr(0)),
])
def test_rope_apply_refuses_overlaps_of_the_two_tensors(lib, k):  # noqa: F811
    assert rope_call(lib, None, None, k) == UNSUPPORTED


@pytest.mark.parametrize("first", [64, 32, 127, 1])
def test_rope_apply_in_place_refuses_parts_that_meet(lib, first):  # noqa: F811
    """q turns values [128, 192) of a tensor in place, k values [first + 64, first + 128) of the same one."""
    k = dict(x=ptr(0) + 2 * first, out=ptr(0) + 2 * first, rot_off=64, head_dim=128)
    assert rope_call(lib, None, dict(x=ptr(0), out=ptr(0)), k) == UNSUPPORTED


@pytest.mark.parametrize("a", [(ptr(0), ptr(1), ptr(1) + 4 * 127), (ptr(0), ptr(1), ptr(1)), (ptr(0), ptr(0) + 12, ptr(2)),
                               (ptr(0), ptr(2), ptr(0) + 8), (ptr(0) + 500, ptr(0), ptr(2))])
def test_rope_table_refuses_overlaps(lib, a):  # noqa: F811
    assert lib.mla_rope_table(ctypes.byref(rope_params()), 4, 64, *a, None) == UNSUPPORTED
    assert lib.mla_rope_last_error()


# 6 tokens x 128 heads, 16 pages, tables of 8 pages: every tensor at a place of its own, with room
APART = {n: ptr(1000 * (i + 1)) for i, n in enumerate((
    "q_nope", "q_rope", "kv_nope", "kv_rope", "kv_scales", "block_table", "act_seqs", "tree_lens", "tree_mask", "out",
    "lse", "workspace"))}
SIZES = dict(q_nope=6 * 128 * 1024, q_rope=6 * 128 * 128, kv_nope=2048 * 1024, kv_rope=2048 * 128, kv_scales=2048 * 16,
             block_table=64, act_seqs=8, tree_lens=8, tree_mask=48, out=6 * 128 * 1024, lse=6 * 128 * 4)
BIG = 1 << 40  # bytes given as workspace; the call needs some 10 MB of them


@pytest.mark.parametrize("written", ["out", "lse", "workspace"])
@pytest.mark.parametrize("other", [n for n in APART if n != "workspace"])
def test_tree_attention_refuses_overlaps(lib, other, written):  # noqa: F811
    if other == written:
        return
    int8 = dict(kv_dtype=1) if other == "kv_scales" else None
    size = SIZES.get(written, 1 << 20)
    for at in (APART[other], APART[other] + -(-SIZES[other] // 256) * 256 - 256, APART[other] - size // 256 * 256 + 256):
        if at >= APART[other] + SIZES[other] or at + size <= APART[other]:
            continue
        assert tree_call(lib, int8, **{**APART, written: at}, nbytes=BIG) == UNSUPPORTED, (other, written, at)
        assert lib.mla_tree_last_error()


# B = 2, S1 = 3, T = 6, W = 4
WRITTEN = dict(block_table=32, act_seqs=8, cache_index=48, positions=24, seq_ids=24, cu_seqs=12, tree_mask=48, num_taken=4)


@pytest.mark.parametrize("first", WRITTEN)
@pytest.mark.parametrize("second", WRITTEN)
def test_page_plan_refuses_outputs_over_one_another(lib, first, second):  # noqa: F811
    if first == second:
        return
    base = ptr(500)
    for at in (base, base + (WRITTEN[first] - 1) // 8 * 8):  # the same place, and the first one's last bytes
        d, io = page_args(**{first: base, second: at})
        assert lib.mla_page_plan(ctypes.byref(d), ctypes.byref(io), None) == UNSUPPORTED, at
        assert lib.mla_page_last_error()


def test_page_plan_takes_an_empty_free_list_from_anywhere(lib):  # noqa: F811
    """A list that has been used up may point into what the step writes: nothing of it is read."""
    d, io = page_args(num_free=0, free_blocks=page_args()[1].block_table + 4)
    assert lib.mla_page_plan(ctypes.byref(d), ctypes.byref(io), None) == -6, lib.mla_page_last_error()  # no device
