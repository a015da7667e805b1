"""Host-side checks of the calls around a drafted decode step: exported
symbols, and bad arguments refused before any CUDA call runs."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from mla_sparse_top_gb300 import build, binding
    build.build()
    return binding.load_library()


def declared(*headers):
    names = set()
    for h in headers:
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h)).read(), flags=re.S)
        names |= set(re.findall(r"\b(mla_\w+)\s*\(", text))
    return names


def test_library_exports_what_the_headers_declare(lib):
    from mla_sparse_top_gb300 import binding
    names = declared("mla_pages.h", "mla_rope.h", "mla_tree.h")
    assert names == set(binding.STEP_SYMBOLS)
    for n in names:
        assert hasattr(lib, n), n


def ptr(i):
    return 0x10000 * (i + 1)


def page_args(**kw):
    from mla_sparse_top_gb300.binding import PageDims, PageIo
    d = dict(B=2, S1=3, T=6, block_size=128, num_blocks=16, max_blocks_per_seq=4, num_free=5)
    io = {n: ptr(i) for i, (n, _) in enumerate(PageIo._fields_)}
    for k, v in kw.items():
        (d if k in d else io)[k] = v
    return PageDims(**d), PageIo(**io)


@pytest.mark.parametrize("change,expect", [
    (dict(B=-1), -2), (dict(S1=-1), -2), (dict(T=7), -2), (dict(T=-6, S1=0, parents=None, tree_mask=None), -2),
    (dict(num_free=-1), -2), (dict(num_blocks=0), -2), (dict(num_blocks=1 << 24), -2),
    (dict(max_blocks_per_seq=0), -2), (dict(block_size=64), -4), (dict(S1=0, T=9), -4),
    (dict(S1=0, T=9, tree_mask=None), -4), (dict(S1=0, T=9, parents=None, tree_mask=None, new_lens=None), -1),
    (dict(B=0, S1=0, T=4, parents=None, tree_mask=None), -2), (dict(ctx_lens=None), -1),
    (dict(block_table=None), -1), (dict(act_seqs=None), -1), (dict(cache_index=None), -1),
    (dict(free_blocks=None), -1), (dict(positions=ptr(3) + 2), -5), (dict(cache_index=ptr(3) + 4), -5),
    (dict(tree_mask=ptr(3) + 4), -5), (dict(num_taken=ptr(3) + 1), -5), (dict(S1=2 ** 30, B=2 ** 30, T=0), -2),
])
def test_page_plan_refuses(lib, change, expect):
    d, io = page_args(**change)
    assert lib.mla_page_plan(ctypes.byref(d), ctypes.byref(io), None) == expect
    assert lib.mla_page_last_error()


def test_page_plan_refuses_outputs_over_inputs(lib):
    for change in (dict(act_seqs=ptr(0)), dict(cache_index=ptr(0)), dict(cu_seqs=ptr(1) + 4), dict(positions=ptr(2)),
                   dict(block_table=ptr(0) + 4), dict(tree_mask=ptr(3) + 16), dict(num_taken=ptr(3) + 20)):
        d, io = page_args(**change)
        assert lib.mla_page_plan(ctypes.byref(d), ctypes.byref(io), None) == -4, change


def test_page_plan_null_structs_and_no_sequences(lib):
    d, io = page_args()
    assert lib.mla_page_plan(None, ctypes.byref(io), None) == -1
    assert lib.mla_page_plan(ctypes.byref(d), None, None) == -1
    d, io = page_args(B=0, T=0)
    assert lib.mla_page_plan(ctypes.byref(d), ctypes.byref(io), None) == 0  # a no-op


def rope_params(**kw):
    from mla_sparse_top_gb300.binding import RopeParams
    p = dict(theta=10000.0, factor=4.0, orig_positions=4096.0, beta_fast=32.0, beta_slow=1.0, mscale=1.0, scaling=3)
    p.update(kw)
    return RopeParams(**p)


@pytest.mark.parametrize("change,rot,T,expect", [
    (dict(theta=1.0), 64, 5, -2), (dict(theta=float("nan")), 64, 5, -2), (dict(theta=float("inf")), 64, 5, -2),
    (dict(factor=0.5), 64, 5, -2), (dict(mscale=1e39), 64, 5, -2), (dict(factor=float("nan")), 64, 5, -2), (dict(mscale=0.0), 64, 5, -2),
    (dict(mscale=float("inf")), 64, 5, -2), (dict(scaling=4), 64, 5, -2), (dict(scaling=-1), 64, 5, -2),
    (dict(orig_positions=0.0), 64, 5, -2), (dict(beta_slow=0.0), 64, 5, -2), (dict(beta_fast=0.5), 64, 5, -2),
    ({}, 0, 5, -2), ({}, 63, 5, -2), ({}, 258, 5, -2), ({}, 64, -1, -2), ({}, 64, 0, 0),
    (dict(scaling=0, factor=0.0), 64, 0, 0),
])
def test_rope_table_refuses(lib, change, rot, T, expect):
    p = rope_params(**change)
    assert lib.mla_rope_table(ctypes.byref(p), T, rot, ptr(0), ptr(1), ptr(2), None) == expect
    assert bool(lib.mla_rope_last_error()) == (expect != 0)


def test_rope_table_pointers(lib):
    p = rope_params()
    assert lib.mla_rope_table(None, 4, 64, ptr(0), ptr(1), ptr(2), None) == -1
    assert lib.mla_rope_table(ctypes.byref(p), 4, 64, None, ptr(1), ptr(2), None) == -1
    assert lib.mla_rope_table(ctypes.byref(p), 4, 64, ptr(0), ptr(1) + 2, ptr(2), None) == -5


def rope_call(lib, dims=None, tensor=None, k=None, positions=ptr(9), params=None):
    from mla_sparse_top_gb300.binding import RopeDims, RopeTensor
    d = dict(T=8, rot_dim=64, half=0, inverse=0, dtype=0)
    d.update(dims or {})
    t = dict(x=ptr(0), out=ptr(1), x_token_stride=4 * 192, x_head_stride=192, out_token_stride=4 * 192,
             out_head_stride=192, rows=None, num_rows=0, n_heads=4, head_dim=192, rot_off=128, reserved=0)
    kt = None if k is None else RopeTensor(**{**t, **k})
    q = RopeTensor(**{**t, **(tensor or {})})
    return lib.mla_rope_apply(ctypes.byref(RopeDims(**d)), ctypes.byref(params or rope_params()), positions,
                              ctypes.byref(q), None if kt is None else ctypes.byref(kt), None)


@pytest.mark.parametrize("dims,tensor,expect", [
    (dict(T=-1), {}, -2), (dict(half=2), {}, -2), (dict(inverse=-1), {}, -2), (dict(dtype=3), {}, -3),
    (dict(dtype=-1), {}, -3), (dict(rot_dim=66), {}, -2), (dict(rot_dim=63), {}, -2), ({}, dict(rot_off=129), -2),
    ({}, dict(rot_off=-1), -2), ({}, dict(n_heads=0), -2), ({}, dict(x=None), -1), ({}, dict(out=None), -1),
    ({}, dict(x=ptr(0) + 1), -5), (dict(dtype=2), dict(out=ptr(1) + 2), -5), ({}, dict(x_token_stride=-1), -2),
    ({}, dict(out_head_stride=191), -2), ({}, dict(out_token_stride=4 * 192 - 1), -2),
    ({}, dict(out_token_stride=192, out_head_stride=192), -2),
    ({}, dict(out_token_stride=192, out_head_stride=8 * 192 - 1), -2),
    ({}, dict(out=ptr(0), out_token_stride=5 * 192), -2), ({}, dict(rows=ptr(5), num_rows=0), -2),
    ({}, dict(rows=ptr(5), num_rows=10, out=ptr(0)), -4), ({}, dict(rows=ptr(5) + 4, num_rows=10), -5),
    ({}, dict(head_dim=(1 << 20) + 8, out_head_stride=1 << 21, out_token_stride=1 << 23), -2),
])
def test_rope_apply_refuses(lib, dims, tensor, expect):
    assert rope_call(lib, dims, tensor) == expect
    assert lib.mla_rope_last_error()
    if tensor:  # the second tensor is checked the same way
        assert rope_call(lib, dims, None, tensor) == expect


def test_rope_apply_pointers_and_no_tokens(lib):
    assert rope_call(lib, positions=None) == -1
    assert rope_call(lib, positions=ptr(9) + 2) == -5
    assert rope_call(lib, dict(T=0), dict(x=None, out=None), positions=None) == 0


def tree_call(lib, dims=None, **kw):
    from mla_sparse_top_gb300.binding import MlaDims
    d = dict(B=2, S1=3, n_q=128, n_kv=1, d_nope=512, d_rope=64, block_size=128, num_blocks=16, max_blocks_per_seq=8,
             topk=0, kv_dtype=0)
    d.update(dims or {})
    names = ("q_nope", "q_rope", "kv_nope", "kv_rope", "kv_scales", "block_table", "act_seqs", "tree_lens",
             "tree_mask", "out", "lse")
    a = {n: ptr(i) for i, n in enumerate(names)}
    a.update(scale=0.04, workspace=ptr(40), nbytes=1 << 40)
    a.update(kw)
    return lib.mla_tree_attn_fwd(ctypes.byref(MlaDims(**d)), *[a[n] for n in names], a["scale"], a["workspace"],
                                 a["nbytes"], None)


@pytest.mark.parametrize("dims,kw,expect", [
    (dict(B=0), {}, -2), (dict(S1=0), {}, -2), (dict(n_q=0), {}, -2), (dict(n_q=129), {}, -2), (dict(n_kv=2), {}, -4),
    (dict(d_nope=256), {}, -4), (dict(d_rope=32), {}, -4), (dict(block_size=64), {}, -4), (dict(num_blocks=0), {}, -2),
    (dict(num_blocks=1 << 24), {}, -2), (dict(max_blocks_per_seq=0), {}, -2), (dict(kv_dtype=2), {}, -3),
    (dict(kv_dtype=1), dict(kv_scales=None), -3), (dict(B=1 << 20, S1=1 << 10, n_q=2), {}, -2),
    ({}, dict(q_nope=None), -1), ({}, dict(q_rope=None), -1), ({}, dict(kv_nope=None), -1), ({}, dict(kv_rope=None), -1),
    ({}, dict(block_table=None), -1), ({}, dict(act_seqs=None), -1), ({}, dict(out=None), -1),
    ({}, dict(workspace=None), -1), ({}, dict(nbytes=1), -2), ({}, dict(scale=float("nan")), -2),
    ({}, dict(scale=float("inf")), -2), ({}, dict(q_nope=ptr(0) + 8), -5), ({}, dict(out=ptr(0) + 8), -5),
    (dict(kv_dtype=1), dict(kv_scales=ptr(0) + 8), -5), ({}, dict(tree_mask=ptr(0) + 4), -5),
    ({}, dict(tree_lens=ptr(0) + 2), -5), ({}, dict(workspace=ptr(40) + 128), -5), ({}, dict(lse=ptr(0) + 2), -5),
])
def test_tree_attention_refuses(lib, dims, kw, expect):
    assert tree_call(lib, dims, **kw) == expect
    assert lib.mla_tree_last_error()


def test_tree_workspace_of_bad_dims_is_zero(lib):
    from mla_sparse_top_gb300.binding import MlaDims
    d = MlaDims(B=2, S1=3, n_q=129, n_kv=1, d_nope=512, d_rope=64, block_size=128, num_blocks=16, max_blocks_per_seq=8)
    assert lib.mla_tree_workspace_bytes(ctypes.byref(d)) == 0 and lib.mla_tree_workspace_bytes(None) == 0
    d.n_q = 128
    assert lib.mla_tree_workspace_bytes(ctypes.byref(d)) > 0
    assert lib.mla_tree_attn_fwd(None, *[None] * 11, 0.0, None, 0, None) == -1
