"""Rotation of views that share their storage without sharing a value: the
overlap check must let them through, and the result must be that of copies."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def turn(positions, q, k=None, **kw):
    import mla_sparse_top_gb300 as mla
    mla.mla_rope_apply(positions, q, k, params=mla.rope_params(), rot_dim=64, **kw)
    torch.cuda.synchronize()


def views(kind, T):
    """(q, its rot_off, k, its rot_off) of one tensor."""
    if kind == "fused":  # queries, keys and values of a token side by side
        x = torch.randn((T, 10, 96), device="cuda").bfloat16()
        return x, x[:, :6], 0, x[:, 6:8], 32
    if kind == "head by head":
        x = torch.randn((T, 8, 96), device="cuda").bfloat16()
        return x, x[:, ::2], 32, x[:, 1::2], 0
    if kind == "heads outermost":
        x = torch.randn((8, T, 64), device="cuda")
        return x, x[:5].transpose(0, 1), 0, x[5:].transpose(0, 1), 0
    if kind == "two parts of a head":
        x = torch.randn((T, 4, 192), device="cuda").half()
        return x, x, 128, x[:, :, :128], 64
    x = torch.randn((2 * T, 3, 64), device="cuda").bfloat16()  # every other token
    return x, x[::2], 0, x[1::2], 0


KINDS = ["fused", "head by head", "heads outermost", "two parts of a head", "every other token"]


@pytest.mark.parametrize("T", [1, 77])
@pytest.mark.parametrize("kind", KINDS)
def test_in_place(kind, T):
    x, q, qo, k, ko = views(kind, T)
    pos = torch.randint(0, 5000, (T,), device="cuda", dtype=torch.int32)
    wq, wk, before = torch.empty_like(q), torch.empty_like(k), x.clone()
    turn(pos, q.clone(), k.clone(), rot_off=qo, k_rot_off=ko, out=wq, k_out=wk)
    turn(pos, q, k, rot_off=qo, k_rot_off=ko)
    assert torch.equal(q[..., qo:qo + 64], wq[..., qo:qo + 64])
    assert torch.equal(k[..., ko:ko + 64], wk[..., ko:ko + 64])
    q[..., qo:qo + 64] = 0
    k[..., ko:ko + 64] = 0
    fresh = before.clone()  # nothing else moved
    a, b = (v if v is not x else fresh for v in (q, k))
    for v, off in ((a, qo), (b, ko)):
        fresh.as_strided(v.shape, v.stride(), v.storage_offset())[..., off:off + 64] = 0
    assert torch.equal(x, fresh)


@pytest.mark.parametrize("T", [1, 77])
@pytest.mark.parametrize("kind", KINDS[:3] + KINDS[4:])
def test_from_one_view_into_the_other(kind, T):
    x, q, qo, k, _ = views(kind, T)
    k = k[:, :q.shape[1]]
    q = q[:, :k.shape[1]]
    pos = torch.randint(0, 5000, (T,), device="cuda", dtype=torch.int32)
    want, source = torch.empty_like(q), q.clone()
    turn(pos, source, rot_off=qo, out=want)
    turn(pos, q, rot_off=qo, out=k)
    assert torch.equal(k, want) and torch.equal(q, source)


def test_the_binding_reports_an_overlap():
    import mla_sparse_top_gb300 as mla
    x = torch.randn((9, 4, 64), device="cuda")
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(mla.MlaError, match="overlap"):
        turn(pos, x[:8], out=x[1:])
    with pytest.raises(mla.MlaError, match="overlap"):
        turn(pos, x[:8], x[1:])
