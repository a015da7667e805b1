"""Host-side checks of the calls on ordinary heads: exported symbols, bad
arguments and overlaps refused before any CUDA call runs, the binding's checks."""
import ctypes
import os

import pytest
import torch

from test_step_abi_host import declared, lib, ptr, rope_params  # noqa: F401
from test_step_limits_host import BF16, F32, I32, I64, Shaped, mla  # noqa: F401

NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN = -1, -2, -3, -4, -5


def test_library_exports_what_the_header_declares(lib):  # noqa: F811
    from mla_sparse_top_gb300 import binding
    assert declared("mla_heads.h") == set(binding.HEADS_SYMBOLS)
    for n in binding.HEADS_SYMBOLS:
        assert hasattr(lib, n), n
    assert os.path.exists(binding.LIB_PATH)


def norm(**kw):
    from mla_sparse_top_gb300.binding import HeadNorm
    d = dict(weight=ptr(20), bias=None, kind=1, fp32=0, eps=1e-6, reserved=0)
    return HeadNorm(**{**d, **kw})


def tensor(i=0, **kw):
    from mla_sparse_top_gb300.binding import RopeTensor
    d = dict(x=ptr(2 * i), out=ptr(2 * i + 1), x_token_stride=512, x_head_stride=128, out_token_stride=512, out_head_stride=128,
             rows=None, num_rows=0, n_heads=4, head_dim=128, rot_off=0, reserved=0)
    return RopeTensor(**{**d, **kw})


def norm_rope(lib, dims={}, params={}, q={}, k=None, qn=None, kn=None, positions=ptr(30)):  # noqa: F811
    from mla_sparse_top_gb300.binding import RopeDims
    d = RopeDims(**{**dict(T=5, rot_dim=64, half=0, inverse=0, dtype=0), **dims})
    p = None if params is None else rope_params(**params)
    return lib.mla_norm_rope(d, p, positions, tensor(**q), None if qn is None else norm(**qn),
                             None if k is None else tensor(1, **k), None if kn is None else norm(**kn), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dims=dict(T=-1)), SHAPE), (dict(dims=dict(rot_dim=3)), SHAPE), (dict(dims=dict(rot_dim=258)), SHAPE),
    (dict(dims=dict(rot_dim=-2)), SHAPE), (dict(dims=dict(half=2)), SHAPE), (dict(dims=dict(inverse=1)), UNSUPPORTED),
    (dict(dims=dict(dtype=3)), DTYPE), (dict(params=None), NULL), (dict(positions=None), NULL), (dict(positions=ptr(30) + 2), ALIGN),
    (dict(q=dict(x=None)), NULL), (dict(q=dict(out=None)), NULL), (dict(q=dict(n_heads=0)), SHAPE), (dict(q=dict(rot_off=65)), SHAPE),
    (dict(q=dict(rot_off=-1)), SHAPE), (dict(q=dict(head_dim=0)), SHAPE), (dict(q=dict(x_head_stride=-128)), SHAPE),
    (dict(q=dict(out_head_stride=64)), SHAPE), (dict(q=dict(out_token_stride=0)), SHAPE), (dict(q=dict(x=ptr(0) + 1)), ALIGN),
    (dict(q=dict(out=ptr(0) + 64)), UNSUPPORTED), (dict(q=dict(out=ptr(30) - 64)), UNSUPPORTED), (dict(q=dict(out=ptr(0), out_token_stride=1024)), SHAPE),
    (dict(qn=dict(kind=3)), SHAPE), (dict(qn=dict(kind=-1)), SHAPE), (dict(qn=dict(eps=-1.0)), SHAPE), (dict(qn=dict(eps=float("nan"))), SHAPE),
    (dict(qn=dict(eps=float("inf"))), SHAPE), (dict(qn=dict(fp32=2)), SHAPE), (dict(qn=dict(bias=ptr(21))), UNSUPPORTED),
    (dict(qn=dict(weight=ptr(20) + 1)), ALIGN), (dict(qn=dict(fp32=1, weight=ptr(20) + 2)), ALIGN), (dict(qn=dict(weight=ptr(1))), UNSUPPORTED),
    (dict(k={}, kn=dict(kind=7)), SHAPE), (dict(k=dict(out=ptr(1))), UNSUPPORTED), (dict(k=dict(rows=ptr(9), num_rows=0)), SHAPE),
    (dict(k=dict(rows=ptr(9) + 4, num_rows=9)), ALIGN), (dict(k=dict(rows=ptr(9), num_rows=9, out=ptr(2))), UNSUPPORTED),
    (dict(k=dict(x=ptr(1) + 256)), UNSUPPORTED),
])
def test_norm_rope_refuses(lib, kw, expect):  # noqa: F811
    assert norm_rope(lib, **kw) == expect
    assert lib.mla_heads_last_error()


def test_norm_rope_no_ops_and_nulls(lib):  # noqa: F811
    from mla_sparse_top_gb300.binding import RopeDims
    assert norm_rope(lib, dims=dict(T=0)) == 0
    assert lib.mla_norm_rope(None, None, None, tensor(), None, None, None, None) == NULL
    assert lib.mla_norm_rope(RopeDims(1, 0, 0, 0, 0), None, None, None, None, None, None, None) == NULL


def append(lib, dims={}, rows=ptr(31), positions=ptr(30), params={}, drop=(), kn=None, q=None, **kw):  # noqa: F811
    from mla_sparse_top_gb300.binding import AppendDims, HeadsTensor, KvCache
    d = dict(T=5, n_kv=2, d_qk=64, d_v=64, rot_dim=64, rot_off=0, half=0, dtype=0, num_blocks=3)
    t = dict(k=HeadsTensor(ptr(0), 128, 64), v=HeadsTensor(ptr(1), 128, 64),
             kc=KvCache(0x4000000, 128 * 128, 128, 64), vc=KvCache(0x5000000, 128 * 128, 128, 64))
    for name, (field, value) in kw.items():
        setattr(t[name], field, value)
    for name in drop:
        t[name] = None
    return lib.mla_kv_append(AppendDims(**{**d, **dims}), None if params is None else rope_params(**params), positions, rows, t["k"],
                             None if kn is None else norm(**kn), t["kc"], t["v"], t["vc"], None if q is None else tensor(4, **q), None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dims=dict(T=-1)), SHAPE), (dict(dims=dict(n_kv=0)), SHAPE), (dict(dims=dict(d_v=0)), SHAPE), (dict(dims=dict(rot_off=2)), SHAPE),
    (dict(dims=dict(num_blocks=0)), SHAPE), (dict(dims=dict(num_blocks=1 << 24)), SHAPE), (dict(dims=dict(dtype=-1)), DTYPE),
    (dict(dims=dict(rot_dim=5)), SHAPE), (dict(dims=dict(half=-1)), SHAPE), (dict(rows=None), NULL), (dict(rows=ptr(31) + 4), ALIGN),
    (dict(positions=None), NULL), (dict(params=None), NULL), (dict(drop=["k"]), NULL), (dict(drop=["vc"]), NULL), (dict(k=("data", None)), NULL),
    (dict(kc=("data", None)), NULL), (dict(kc=("row_stride", 64)), SHAPE), (dict(kc=("block_stride", 128)), SHAPE), (dict(vc=("head_stride", 0)), SHAPE),
    (dict(vc=("data", 0x4000000)), UNSUPPORTED), (dict(kc=("data", 0x4000001)), ALIGN), (dict(v=("data", 0x5000000)), UNSUPPORTED),
    (dict(kn=dict(kind=9)), SHAPE), (dict(kn=dict(weight=0x4000100)), UNSUPPORTED), (dict(q=dict(rows=ptr(9), num_rows=5)), UNSUPPORTED),
    (dict(q=dict(out=0x4000000)), UNSUPPORTED), (dict(q=dict(out=ptr(0))), UNSUPPORTED),
])
def test_append_refuses(lib, kw, expect):  # noqa: F811
    assert append(lib, **kw) == expect
    assert lib.mla_heads_last_error()


def test_append_no_op(lib):  # noqa: F811
    assert append(lib, dims=dict(T=0), rows=None) == 0


def prompt(lib, dims={}, nulls=(), ws=None, scale=0.1, **kw):  # noqa: F811
    from mla_sparse_top_gb300.binding import HeadsTensor, KvCache, PromptDims
    d = PromptDims(**{**dict(B=2, T=10, Tk=10, n_q=4, n_kv=2, d_qk=64, d_v=64, dtype=0, causal=1, num_blocks=0, max_blocks_per_seq=0), **dims})
    need = lib.mla_prompt_workspace_bytes(d)
    a = dict(q=HeadsTensor(0x1000000, 256, 64), k=KvCache(0x2000000, 0, 128, 64), v=KvCache(0x3000000, 0, 128, 64), cu_q=ptr(1), cu_k=None,
             table=None, act=None, out=0x4000000, lse=0x5000000, work=0x40000000)
    if d.num_blocks > 0:
        a.update(k=KvCache(0x2000000, 128 * 128, 128, 64), v=KvCache(0x3000000, 128 * 128, 128, 64), table=ptr(2), act=ptr(3))
    for name, value in kw.items():
        if isinstance(value, tuple):
            setattr(a[name], *value)
        else:
            a[name] = value
    for name in nulls:
        a[name] = None
    return lib.mla_prompt_attn_fwd(d, a["q"], a["k"], a["v"], a["cu_q"], a["cu_k"], a["table"], a["act"], a["out"], a["lse"], scale, a["work"],
                                   need if ws is None else ws, None)


PAGED = dict(Tk=0, num_blocks=4, max_blocks_per_seq=3)


@pytest.mark.parametrize("kw,expect", [
    (dict(dims=dict(B=-1)), SHAPE), (dict(dims=dict(T=-1)), SHAPE), (dict(dims=dict(Tk=-1)), SHAPE), (dict(dims=dict(n_q=5)), SHAPE),
    (dict(dims=dict(n_kv=0)), SHAPE), (dict(dims=dict(n_q=129, n_kv=1)), UNSUPPORTED), (dict(dims=dict(d_qk=60)), SHAPE),
    (dict(dims=dict(d_v=0)), SHAPE), (dict(dims=dict(d_qk=200)), UNSUPPORTED), (dict(dims=dict(d_v=136)), UNSUPPORTED),
    (dict(dims=dict(dtype=2)), DTYPE), (dict(dims=dict(causal=2)), SHAPE), (dict(dims=dict(num_blocks=1 << 24)), SHAPE),
    (dict(dims=dict(num_blocks=4)), SHAPE), (dict(dims=dict(max_blocks_per_seq=4)), SHAPE), (dict(dims=dict(T=1 << 30, n_q=4)), SHAPE),
    (dict(dims=dict(PAGED, max_blocks_per_seq=(1 << 23) + 1)), SHAPE), (dict(nulls=["q"]), NULL), (dict(nulls=["k"]), NULL),
    (dict(q=("data", None)), NULL), (dict(v=("data", None)), NULL), (dict(nulls=["cu_q"]), NULL), (dict(nulls=["out"]), NULL),
    (dict(dims=PAGED, nulls=["table"]), NULL), (dict(dims=PAGED, nulls=["act"]), NULL), (dict(dims=PAGED, cu_k=ptr(4)), UNSUPPORTED),
    (dict(table=ptr(2)), UNSUPPORTED), (dict(act=ptr(2)), UNSUPPORTED), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(q=("token_stride", -256)), SHAPE), (dict(q=("head_stride", 60)), ALIGN), (dict(k=("row_stride", 1 << 39)), SHAPE),
    (dict(q=("data", 0x1000008)), ALIGN), (dict(out=0x4000008), ALIGN), (dict(cu_q=ptr(1) + 2), ALIGN), (dict(lse=0x5000002), ALIGN),
    (dict(work=0x40000080), ALIGN), (dict(out=0x1000000), UNSUPPORTED), (dict(out=0x2000100), UNSUPPORTED), (dict(lse=0x3000100), UNSUPPORTED),
    (dict(lse=0x4000010), UNSUPPORTED), (dict(work=0x4000000), UNSUPPORTED), (dict(out=ptr(1)), UNSUPPORTED),
    (dict(dims=PAGED, out=0x2000000), UNSUPPORTED), (dict(dims=PAGED, lse=ptr(2)), UNSUPPORTED),
])
def test_prompt_refuses(lib, kw, expect):  # noqa: F811
    assert prompt(lib, **kw) == expect
    assert lib.mla_heads_last_error()


def test_prompt_no_ops_and_small_workspace(lib):  # noqa: F811
    from mla_sparse_top_gb300.binding import PromptDims
    assert prompt(lib, dims=dict(B=0)) == 0 and prompt(lib, dims=dict(T=0)) == 0
    assert prompt(lib, ws=8) == SHAPE
    assert lib.mla_prompt_workspace_bytes(None) == 0
    assert lib.mla_prompt_workspace_bytes(PromptDims(1, 1, 1, 3, 2, 64, 64, 0, 1, 0, 0)) == 0


def paged(lib, dims={}, nulls=(), ws=None, **kw):  # noqa: F811
    from mla_sparse_top_gb300.binding import HeadsTensor, KvCache, PagedDims
    d = PagedDims(**{**dict(B=2, S1=1, n_q=4, n_kv=2, d_qk=64, d_v=64, dtype=0, num_blocks=4, max_blocks_per_seq=3), **dims})
    need = lib.mla_paged_workspace_bytes(d)
    a = dict(q=HeadsTensor(0x1000000, 256, 64), k=KvCache(0x2000000, 128 * 128, 128, 64), v=KvCache(0x3000000, 128 * 128, 128, 64), table=ptr(2),
             act=ptr(3), lens=ptr(4), out=0x4000000, lse=0x5000000, work=0x40000000)
    for name, value in kw.items():
        if isinstance(value, tuple):
            setattr(a[name], *value)
        else:
            a[name] = value
    for name in nulls:
        a[name] = None
    return lib.mla_paged_attn_fwd(d, a["q"], a["k"], a["v"], a["table"], a["act"], a["lens"], a["out"], a["lse"], 0.1, a["work"],
                                  need if ws is None else ws, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dims=dict(B=-1)), SHAPE), (dict(dims=dict(S1=0)), SHAPE), (dict(dims=dict(S1=(1 << 20) + 1)), SHAPE), (dict(dims=dict(n_q=3)), SHAPE),
    (dict(dims=dict(d_qk=4)), SHAPE), (dict(dims=dict(d_v=256)), UNSUPPORTED), (dict(dims=dict(dtype=5)), DTYPE), (dict(dims=dict(num_blocks=0)), SHAPE),
    (dict(dims=dict(max_blocks_per_seq=0)), SHAPE), (dict(dims=dict(B=1 << 15, S1=1 << 15)), SHAPE), (dict(nulls=["q"]), NULL), (dict(nulls=["table"]), NULL),
    (dict(nulls=["act"]), NULL), (dict(nulls=["out"]), NULL), (dict(k=("data", None)), NULL), (dict(v=("data", 0x3000004)), ALIGN),
    (dict(k=("block_stride", 1 << 40)), SHAPE), (dict(v=("row_stride", 100)), ALIGN), (dict(lens=ptr(4) + 1), ALIGN), (dict(act=ptr(3) + 2), ALIGN),
    (dict(out=0x2000000), UNSUPPORTED), (dict(lse=0x4000000), UNSUPPORTED), (dict(out=ptr(4)), UNSUPPORTED), (dict(ws=8), SHAPE),
])
def test_paged_refuses(lib, kw, expect):  # noqa: F811
    assert paged(lib, **kw) == expect
    assert lib.mla_heads_last_error()


def test_paged_no_op(lib):  # noqa: F811
    assert paged(lib, dims=dict(B=0)) == 0
    assert lib.mla_paged_workspace_bytes(None) == 0


@pytest.mark.parametrize("over", [1 << 31, (1 << 32) + 8])
def test_binding_refuses_sizes_beyond_32_bits(mla, over):  # noqa: F811
    table = Shaped(I32, 2, 3)
    for q, k, b in (((over, 4, 64), (8, 2, 64), None), ((8, over, 64), (8, 2, 64), None), ((8, 4, 64), (over, 2, 64), None),
                    ((8, 4, 64), (over, 128, 2, 64), table), ((8, 4, 64), (9, 128, 2, 64), Shaped(I32, 2, over))):
        with pytest.raises(ValueError, match="32 bits"):
            mla.prompt_dims(Shaped(BF16, *q), Shaped(BF16, *k), Shaped(BF16, *k), Shaped(I32, 3), block_table=b)
    for q, k, b in (((over, 4, 64), (9, 128, 2, 64), 3), ((2, 4, 64), (over, 128, 2, 64), 3), ((2, 4, 64), (9, 128, 2, 64), over)):
        with pytest.raises(ValueError, match="32 bits"):
            mla.paged_dims(Shaped(BF16, *q), Shaped(BF16, *k), Shaped(BF16, *k), Shaped(I32, 2, b), S1=1)
    for T, rot in ((over, 0), (4, over)):
        with pytest.raises(ValueError, match="32 bits"):
            mla.mla_norm_rope(Shaped(I32, T), Shaped(BF16, T, 2, 64), rot_dim=rot)


def test_binding_refuses_wrong_types_and_shapes(mla):  # noqa: F811
    with pytest.raises(ValueError):
        mla.mla_norm_rope(None, Shaped(I64, 4, 2, 64))
    with pytest.raises(ValueError):
        mla.prompt_dims(Shaped(F32, 8, 4, 64), Shaped(F32, 8, 2, 64), Shaped(F32, 8, 2, 64), Shaped(I32, 3))
    with pytest.raises(ValueError):
        mla.paged_dims(Shaped(BF16, 7, 4, 64), Shaped(BF16, 9, 128, 2, 64), Shaped(BF16, 9, 128, 2, 64), Shaped(I32, 2, 3), S1=2)
    with pytest.raises(ValueError):
        mla.head_norm("rms", torch.ones(4))
    with pytest.raises(KeyError):
        mla.head_norm("batch")


def test_oracle_of_the_norms_and_attention():
    """The oracle against closed forms."""
    import numpy as np

    from oracle import heads
    x = np.array([[[3.0, 4.0]]])
    assert np.allclose(heads.norm(x, "rms", eps=0), x / np.sqrt(12.5))
    assert np.allclose(heads.norm(x, "layer", np.array([2.0, 1.0]), np.array([1.0, 0.0]), eps=0.75), [[[0.0, 0.5]]])
    q, k, v = np.ones((2, 2, 4)), np.ones((3, 1, 4)), np.arange(3.0).reshape(3, 1, 1)
    out, lse, mass, terms, top = heads.attention(q, k, v, 0.5, True)
    assert np.allclose(out[:, 0, 0], [0.5, 1.0]) and np.allclose(lse[:, 1], [2 + np.log(2), 2 + np.log(3)])
    assert np.allclose(mass, out) and (terms == 2).all() and (top == 2).all()
    out, lse = heads.attention(q, k[:1], v[:1], 0.5, True)[:2]  # fewer keys than queries: the first sees none
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all() and np.isfinite(lse[1]).all()
    assert ctypes.sizeof(ctypes.c_void_p) == 8
