"""Two tensors of which one, both or none have 16-byte aligned rows: each gives
the bits that it gives alone, in one call."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q_pad,k_pad", [(0, 0), (0, 3), (5, 0), (5, 3)])
@pytest.mark.parametrize("T,to_rows,in_place", [(1, False, False), (70, False, False), (70, True, False), (70, False, True)])
def test_tensors_of_different_alignment(T, to_rows, in_place, q_pad, k_pad, dtype, half):
    import mla_sparse_top_gb300 as mla
    g = torch.Generator(device="cuda").manual_seed(T)
    q = torch.randn((T, 6, 96 + q_pad), generator=g, device="cuda").to(dtype)[:, :, :96]
    k = torch.randn((T, 1, 64 + k_pad), generator=g, device="cuda").to(dtype)[:, :, :64]
    pos = torch.randint(0, 9000, (T,), generator=g, device="cuda", dtype=torch.int32)
    rows = torch.randperm(3 * T, generator=g, device="cuda")[:T].contiguous() if to_rows else None
    kw = dict(params=mla.rope_params(), rot_dim=64, half=half)
    wq, wk = torch.zeros_like(q), torch.zeros((3 * T if to_rows else T, 1, 64), dtype=dtype, device="cuda")
    mla.mla_rope_apply(pos, q, rot_off=32, out=wq, **kw)
    alone = torch.zeros_like(k)
    mla.mla_rope_apply(pos, k, out=alone, **kw)
    wk[rows if to_rows else slice(None)] = alone
    if in_place:
        mla.mla_rope_apply(pos, q, k, rot_off=32, **kw)
        assert torch.equal(q, wq) and torch.equal(k, wk)
        return
    oq, ok = torch.zeros_like(q), torch.zeros_like(wk)
    mla.mla_rope_apply(pos, q, k, rot_off=32, out=oq, k_out=ok, k_rows=rows, **kw)
    assert torch.equal(oq, wq) and torch.equal(ok, wk)


def test_strides_that_are_never_taken():
    """One token, one head: whatever their strides say."""
    import mla_sparse_top_gb300 as mla
    x = torch.randn((1, 1, 128), device="cuda").bfloat16()
    pos = torch.tensor([77], dtype=torch.int32, device="cuda")
    want, out = torch.empty_like(x), torch.empty_like(x)
    kw = dict(params=mla.rope_params(), rot_dim=64)
    mla.mla_rope_apply(pos, x, out=want, **kw)
    mla.mla_rope_apply(pos, x.as_strided((1, 1, 128), (1001, 333, 1)), out=out.as_strided((1, 1, 128), (7, 131, 1)), **kw)
    assert torch.equal(out, want)


def test_mixed_alignment_in_a_graph():
    import mla_sparse_top_gb300 as mla
    q = torch.randn((40, 4, 128), device="cuda").bfloat16()
    k = torch.randn((40, 1, 67), device="cuda").bfloat16()[:, :, :64]
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    kw = dict(params=mla.rope_params(), rot_dim=64)
    wq, wk, oq, ok = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(q), torch.zeros_like(k)
    mla.mla_rope_apply(pos, q, k, out=wq, k_out=wk, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_rope_apply(pos, q, k, out=oq, k_out=ok, **kw)
    for _ in range(2):
        oq.zero_(), ok.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oq, wq) and torch.equal(ok, wk)
