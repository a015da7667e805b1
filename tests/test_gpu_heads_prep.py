"""Norms and rotation of heads, and the paged append, on the GPU against the fp64 oracle.

Bound of one output, with u = 2^-24: a sum over a head's D values goes through at most D / 32 + 24
additions, so the mean is off by n u mean|x| (n that number) and a difference c from it by e = n u
mean|x| + u |c|; the mean square by a factor of n u, and by 2 e / s where the c are off (s the root
below the quotient); root, quotient, products and the sum with the bias add 6 u.  Then the rotation
(test_gpu_rope.py): cosines off by 8 u mscale in all, two products, the frequency's |p| 2^-45.  At the end half a
step of the output's type."""
import numpy as np
import pytest
import torch

from heads_util import TYPES, U, cache, np64
from oracle import heads, step

pytestmark = pytest.mark.gpu
SCHEMES = [dict(), dict(scaling="linear", factor=8.0), dict(scaling="yarn", factor=40.0, mscale=1.3688879454113936)]


def norm_bound(x, kind, weight, bias, eps):
    """The normed heads and how far each value may be off before the rotation."""
    y = heads.norm(x, kind, weight, bias, eps)
    if kind is None:
        return y, np.zeros_like(y)
    D = x.shape[-1]
    n = D / 32 + 24
    c = x - x.mean(-1, keepdims=True) if kind == "layer" else x
    e = (n * U * np.abs(x).mean(-1, keepdims=True) + U * np.abs(c)) if kind == "layer" else np.zeros_like(x)
    s = np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    w = 1 if weight is None else np.abs(weight)
    rel = n * U + 2 * e.max(-1, keepdims=True) / s + 6 * U
    return y, w * (e + np.abs(c) * rel) / s + 6 * U * (np.abs(y) + (0 if bias is None else np.abs(bias)))


def want(x, positions, norm, scheme, *, rot_dim, rot_off, half):
    """Expected values and bounds; norm (kind, weight, bias, eps) or None."""
    a = np64(x)
    kind, weight, bias, eps = (None, None, None, 0) if norm is None else norm
    weight, bias = (None if t is None else np64(t) for t in (weight, bias))
    y, b = norm_bound(a, kind, weight, bias, eps)
    if rot_dim:
        sch = dict(scheme)
        ms = sch.pop("mscale", 1.0)
        p = np64(positions)
        n, part = rot_dim // 2, np.abs(y[:, :, rot_off:rot_off + rot_dim])
        off = b[:, :, rot_off:rot_off + rot_dim]
        pair = (lambda t: np.concatenate([t[..., :n] + t[..., n:]] * 2, -1)) if half else \
            (lambda t: np.repeat(t[..., 0::2] + t[..., 1::2], 2, -1))
        y = step.rope_apply(y, p, step.rope_freqs(rot_dim, **sch), rot_off=rot_off, half=half, inverse=False, mscale=ms)
        b = b.copy()
        b[:, :, rot_off:rot_off + rot_dim] = ms * (pair(off) * 1.001 + pair(part) * (10 * U + np.abs(p)[:, None, None] * 2.0 ** -45))
    info = torch.finfo(x.dtype)
    return y, b * 1.001 + np.maximum(np.abs(y), info.smallest_normal) * info.eps / 2 * (1 + 1e-6)


def check(got, x, positions, norm, scheme, what="", **kw):
    y, bound = want(x, positions, norm, scheme, **kw)
    err = np.abs(np64(got) - y)
    assert (err <= bound).all(), f"{what} worst {np.nanmax(err / bound)}"


def inputs(T, H, D, dtype, pad=0, seed=0, maxpos=1 << 17):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, H, D + pad), generator=g) * 2 + 0.3).to(dtype).cuda()[:, :, :D]
    return x, torch.randint(0, maxpos, (T,), generator=g, dtype=torch.int32).cuda()


def make_norm(kind, D, dtype, fp32, seed=0, eps=1e-6):
    """(the oracle's form, the library's)."""
    import mla_sparse_top_gb300 as mla
    if kind is None:
        return None, None
    g = torch.Generator().manual_seed(seed + 100)
    t = torch.float32 if fp32 else dtype
    weight = (torch.randn((D,), generator=g) + 1).to(t).cuda()
    bias = torch.randn((D,), generator=g).to(t).cuda() if kind == "layer" else None
    return (kind, weight, bias, eps), mla.head_norm(kind, weight, bias, eps=eps)


SHAPES = [(1, 1, 64, 0, 64, 0), (1, 32, 128, 0, 128, 0), (33, 5, 192, 128, 64, 0), (7, 3, 107, 7, 36, 5), (100, 1, 2, 0, 2, 0),
          (5, 2, 300, 20, 256, 4), (9, 5, 128, 64, 16, 8), (300, 40, 96, 0, 96, 0), (3, 9, 1000, 8, 64, 0), (2, 3, 2500, 0, 128, 0),
          (4, 2, 1111, 3, 30, 1), (1200, 20, 64, 0, 0, 0), (6, 400, 24, 8, 16, 0), (3, 2, 1, 0, 0, 0), (700, 16, 128, 0, 64, 0),
          (40, 6, 96, 0, 30, 0), (900, 12, 64, 6, 20, 8), (5, 2, 128, 122, 6, 0), (3, 4, 48, 9, 14, 0), (21, 3, 600, 10, 202, 8)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", [None, "rms", "layer"])
@pytest.mark.parametrize("T,H,D,off,rot,pad", SHAPES)
def test_norm_rope(T, H, D, off, rot, pad, kind, dtype):
    import mla_sparse_top_gb300 as mla
    x, pos = inputs(T, H, D, TYPES[dtype], pad, seed=T + D)
    sch = SCHEMES[(T + H + D) % len(SCHEMES)]
    for half in (False, True):
        norm, own = make_norm(kind, D, x.dtype, fp32=half, seed=D)
        kw = dict(rot_dim=rot, rot_off=off, half=half)
        y = torch.full((T, H, D), float("nan"), dtype=x.dtype, device="cuda")
        mla.mla_norm_rope(pos, x, params=mla.rope_params(**sch), out=y, q_norm=own, **kw)
        check(y, x, pos, norm, sch, **kw)
        # in place, between values that stay
        whole = torch.full((T, H, D + pad + 8), 3.0, dtype=x.dtype, device="cuda")
        z = whole[:, :, :D]
        z.copy_(x)
        mla.mla_norm_rope(pos, z, params=mla.rope_params(**sch), q_norm=own, **kw)
        check(z, x, pos, norm, sch, "in place", **kw)
        assert (whole[:, :, D:] == 3).all()
    assert mla.heads_device_status(clear=True) == 0


@pytest.mark.parametrize("q_kind,k_kind,pad", [(None, "layer", 0), ("rms", "rms", 0), ("rms", None, 3), ("layer", "rms", 3)])
def test_queries_and_keys_into_rows(q_kind, k_kind, pad):
    """Index queries and keys: the keys to their cache rows, one skipped, one bad."""
    import mla_sparse_top_gb300 as mla
    T, H, K, D = 37, 16, 2, 128
    q, pos = inputs(T, H, D, torch.bfloat16, pad)
    k, _ = inputs(T, K, D, torch.bfloat16, 0, seed=5)
    qn, qo = make_norm(q_kind, D, q.dtype, True)
    kn, ko = make_norm(k_kind, D, q.dtype, False, seed=3)
    rows = torch.randperm(300)[:T]
    rows[3], rows[5] = -1, 300
    rows_gpu = rows.cuda()
    k_out = torch.full((300, K, D), 5.0, dtype=q.dtype, device="cuda")
    q_out = torch.empty((T, H, D), dtype=q.dtype, device="cuda")
    kw = dict(rot_dim=64, rot_off=0, half=True)
    mla.mla_norm_rope(pos, q, k, params=mla.rope_params(), q_norm=qo, k_norm=ko, out=q_out, k_out=k_out, k_rows=rows_gpu,
                      rot_dim=64, half=True)
    assert mla.heads_device_status(clear=True) == mla.MLA_DEVICE_BAD_BLOCK
    check(q_out, q, pos, qn, {}, "q", **kw)
    live = [t for t in range(T) if 0 <= rows[t] < 300]
    check(k_out[rows_gpu[live]], k[live], pos[live], kn, {}, "k", **kw)
    rest = torch.ones(300, dtype=torch.bool)
    rest[rows[live]] = False
    assert (k_out[rest.cuda()] == 5).all()


@pytest.mark.parametrize("layout", ["token", "head", "shared"])
@pytest.mark.parametrize("T,H,Hkv,D,Dv,rot,dtype,kind,pad", [
    (1, 4, 1, 128, 128, 128, "bf16", "rms", 0), (64, 32, 8, 128, 128, 64, "bf16", "rms", 0), (200, 10, 5, 80, 72, 40, "fp16", None, 0),
    (33, 3, 3, 192, 128, 64, "bf16", "layer", 8), (19, 7, 1, 61, 35, 20, "fp32", "rms", 3), (500, 0, 2, 64, 64, 0, "bf16", None, 0),
    (77, 6, 2, 100, 100, 100, "bf16", "layer", 2)])
def test_append(T, H, Hkv, D, Dv, rot, dtype, kind, pad, layout):
    import mla_sparse_top_gb300 as mla
    dt = TYPES[dtype]
    k, pos = inputs(T, Hkv, D, dt, pad)
    v, _ = inputs(T, Hkv, Dv, dt, pad, seed=1)
    blocks = 2 + T // 64
    kc, vc = cache(blocks, Hkv, D, layout, dt, fill=5.0), cache(blocks, Hkv, Dv, layout, dt, fill=6.0)
    rows = torch.randperm(blocks * 128)[:T]
    bad = T > 20
    if bad:
        rows[3], rows[5], rows[7] = -1, blocks * 128, -(1 << 40)
    norm, own = make_norm(kind, D, dt, True)
    q = q_out = qn = qo = None
    if H:
        q, _ = inputs(T, H, D, dt, pad, seed=2)
        q_out = torch.empty((T, H, D), dtype=dt, device="cuda")
        qn, qo = make_norm(kind, D, dt, False, seed=7)
    mla.mla_kv_append(pos, rows.cuda(), k, v, kc, vc, params=mla.rope_params(), rot_dim=rot, half=True, k_norm=own, q=q,
                      q_out=q_out, q_norm=qo)
    assert mla.heads_device_status(clear=True) == (mla.MLA_DEVICE_BAD_BLOCK if bad else 0)
    live = [t for t in range(T) if 0 <= rows[t] < blocks * 128]
    at = rows[live].cuda()
    kw = dict(rot_dim=rot, rot_off=0, half=True)
    check(kc[at // 128, at % 128], k[live], pos[live], norm, {}, "k", **kw)
    assert torch.equal(vc[at // 128, at % 128], v[live])
    rest = torch.ones((blocks, 128), dtype=torch.bool, device="cuda")
    rest[at // 128, at % 128] = False
    assert (kc[rest] == 5).all() and (vc[rest] == 6).all()
    if H:
        check(q_out, q, pos, qn, {}, "q", **kw)


def test_append_in_place_from_one_fused_tensor():
    """Queries, keys and values as one projection leaves them, the queries turned where they lie."""
    import mla_sparse_top_gb300 as mla
    T, H, Hkv, D = 130, 8, 2, 64
    x = torch.randn((T, (H + 2 * Hkv) * D), dtype=torch.float32).to(torch.bfloat16).cuda()
    old = x.clone()
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split((H * D, Hkv * D, Hkv * D), 1))
    q0, k0, v0 = (t.unflatten(1, (-1, D)) for t in old.split((H * D, Hkv * D, Hkv * D), 1))
    pos = torch.arange(T, dtype=torch.int32).cuda()
    kc, vc = (cache(2, Hkv, D, "token", x.dtype, fill=0.0) for _ in range(2))
    norm, own = make_norm("rms", D, x.dtype, False)
    mla.mla_kv_append(pos, torch.arange(T).cuda(), k, v, kc, vc, params=mla.rope_params(), rot_dim=D, k_norm=own, q=q, q_norm=own)
    kw = dict(rot_dim=D, rot_off=0, half=False)
    check(q, q0, pos, norm, {}, "q", **kw)
    check(kc.flatten(0, 1)[:T], k0, pos, norm, {}, "k", **kw)
    assert torch.equal(vc.flatten(0, 1)[:T], v0) and torch.equal(k, k0) and torch.equal(v, v0)


def test_zero_and_large_heads_and_nan():
    import mla_sparse_top_gb300 as mla
    x, pos = inputs(6, 3, 128, torch.bfloat16)
    x[0] = 0
    x[1] *= 1e15
    x[2, 1, 5] = float("nan")
    for kind in ("rms", "layer"):
        norm, own = make_norm(kind, 128, x.dtype, True)
        y = torch.empty_like(x)
        mla.mla_norm_rope(None, x, q_norm=own, out=y)
        live = torch.ones((6, 3), dtype=torch.bool)
        live[2, 1] = False
        assert torch.isnan(y[2, 1]).all()
        # one token at a time keeps the oracle's arrays dense
        got, ref = y.flatten(0, 1)[live.flatten().cuda()][:, None], x.flatten(0, 1)[live.flatten().cuda()][:, None]
        check(got, ref, pos[:1].expand(17), norm, {}, kind, rot_dim=0, rot_off=0, half=False)


def test_far_positions_and_many_tokens():
    import mla_sparse_top_gb300 as mla
    T = 70000
    x, pos = inputs(T, 1, 64, torch.bfloat16, maxpos=1 << 30)
    norm, own = make_norm("rms", 64, x.dtype, True)
    y = torch.empty_like(x)
    mla.mla_norm_rope(pos, x, params=mla.rope_params(), rot_dim=64, half=True, q_norm=own, out=y)
    for part in (slice(0, 500), slice(T - 500, T)):
        check(y[part], x[part], pos[part], norm, {}, rot_dim=64, rot_off=0, half=True)
