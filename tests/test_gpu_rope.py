"""Rotary positions on the GPU against the fp64 oracle.

Bound of one output, with u = 2^-24 (half a step of fp32): cos and sin are off
by at most 2 ulp of their own, pi u from the angle's rounding to
fp32 (a fraction of a turn below 1/2, relative error u), 2 u from mscale and
its product: below 8 u mscale together; the rotation adds 2 u per term.  So
|error| <= 10 u mscale (|x_a| + |x_b|), plus the frequency's own error |p|
2^-48 turns (2^-45 as an angle), plus half a step of the output's type."""
import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SCHEMES = [dict(), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0, theta=500000.0),
           dict(scaling="yarn", factor=40.0, mscale=1.3688879454113936), dict(scaling="yarn", factor=1.0)]


def want_and_bound(x, positions, scheme, *, rot_dim, rot_off, half, inverse=False):
    sch = dict(scheme)
    m = sch.pop("mscale", 1.0)
    f = step.rope_freqs(rot_dim, **sch)
    a = x.double().cpu().numpy()
    p = positions.cpu().numpy()
    y = step.rope_apply(a, p, f, rot_off=rot_off, half=half, inverse=inverse, mscale=m)
    part = np.abs(a[:, :, rot_off:rot_off + rot_dim])
    n = rot_dim // 2
    if half:
        pair = np.concatenate([part[..., :n] + part[..., n:]] * 2, -1)
    else:
        pair = np.repeat(part[..., 0::2] + part[..., 1::2], 2, -1)
    bound = np.zeros_like(y)
    bound[:, :, rot_off:rot_off + rot_dim] = pair * m * (10 * U + np.abs(p)[:, None, None] * 2.0 ** -45)
    # half a step; below the type's normal range a step is that of its smallest normal number
    info = torch.finfo(x.dtype)
    return y, bound + np.maximum(np.abs(y), info.smallest_normal) * info.eps / 2 * (1 + 1e-6)


def check(got, x, positions, scheme, **kw):
    y, bound = want_and_bound(x, positions, scheme, **kw)
    err = np.abs(got.double().cpu().numpy() - y)
    assert (err <= bound).all(), f"worst {np.nanmax(err / bound)}"
    lo, hi = kw["rot_off"], kw["rot_off"] + kw["rot_dim"]
    assert torch.equal(got[..., :lo], x[..., :lo]) and torch.equal(got[..., hi:], x[..., hi:])


def inputs(T, H, D, dtype, pad=0, maxpos=1 << 17, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D + pad), generator=g).to(dtype).cuda()[:, :, :D]
    return x, torch.randint(0, maxpos, (T,), generator=g, dtype=torch.int32).cuda()


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("rot_dim", [2, 64, 256])
def test_table(scheme, rot_dim):
    import mla_sparse_top_gb300 as mla
    pos = torch.tensor([0, 1, 2, 4095, 4096, 163840, (1 << 20) - 1, -3, 2 ** 24 + 1, 2 ** 31 - 1], dtype=torch.int32)
    c, s = torch.full((2, len(pos), rot_dim // 2), float("nan"), device="cuda")
    mla.mla_rope_table(pos.cuda(), c, s, params=mla.rope_params(**scheme))
    sch = dict(scheme)
    m = sch.pop("mscale", 1.0)
    # the exact angle modulo a turn in extended precision: the oracle's fp64 product is itself off far out
    f = step.rope_freqs(rot_dim, **sch)
    ang = np.array([[np.longdouble(int(p)) * np.longdouble(v) for v in f] for p in pos])
    bound = m * (8 * U + np.abs(pos.numpy().astype(float))[:, None] * 2.0 ** -45)
    assert (np.abs(c.double().cpu().numpy() - m * np.cos(ang).astype(float)) <= bound).all()
    assert (np.abs(s.double().cpu().numpy() - m * np.sin(ang).astype(float)) <= bound).all()


@pytest.mark.parametrize("T", [1, 3, 5000])
def test_table_lengths(T):
    import mla_sparse_top_gb300 as mla
    _, pos = inputs(T, 1, 2, torch.float32)
    c, s = torch.empty((2, T, 32), device="cuda")
    mla.mla_rope_table(pos, c, s, params=mla.rope_params())
    f = step.rope_freqs(64)
    ang = pos.cpu().numpy()[:, None] * f
    bound = 8 * U + (1 << 17) * 2.0 ** -45
    assert np.abs(c.cpu().numpy() - np.cos(ang)).max() <= bound and np.abs(s.cpu().numpy() - np.sin(ang)).max() <= bound


@pytest.mark.parametrize("T,pairs,shift", [(777, 32, 1), (777, 32, 4), (1, 128, 0), (513, 128, 3), (65, 1, 0), (1000, 6, 0),
                                           (300, 100, 0), (129, 4, 0), (31, 127, 2)])
def test_table_widths(T, pairs, shift):
    """Rows in 16-byte stores and without, no value beside them touched."""
    import mla_sparse_top_gb300 as mla
    _, pos = inputs(T, 1, 2, torch.float32, seed=pairs)
    c, s = (torch.full((T * pairs + 8,), -7.0, device="cuda") for _ in range(2))
    mla.mla_rope_table(pos, c[shift:shift + T * pairs].view(T, pairs), s[shift:shift + T * pairs].view(T, pairs),
                       params=mla.rope_params())
    ang = pos.cpu().numpy()[:, None] * step.rope_freqs(2 * pairs)
    bound = 8 * U + (1 << 17) * 2.0 ** -45
    for got, want in ((c, np.cos(ang)), (s, np.sin(ang))):
        got = got.cpu().numpy()
        assert np.abs(got[shift:shift + T * pairs].reshape(T, pairs) - want).max() <= bound
        assert (got[:shift] == -7).all() and (got[shift + T * pairs:] == -7).all()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H,D,rot_off,rot_dim,pad", [
    (1, 1, 64, 0, 64, 0), (1, 128, 192, 128, 64, 0), (33, 64, 128, 0, 64, 0), (7, 3, 107, 7, 36, 5),
    (100, 1, 2, 0, 2, 0), (5, 2, 300, 20, 256, 4), (9, 5, 128, 64, 16, 8), (11, 4, 80, 8, 40, 0), (700, 2, 64, 0, 64, 0),
    (3, 400, 24, 8, 16, 0)])
def test_apply_out_of_place_and_in_place(T, H, D, rot_off, rot_dim, pad, dtype, half):
    import mla_sparse_top_gb300 as mla
    x, pos = inputs(T, H, D, TYPES[dtype], pad, seed=T + H)
    sch = SCHEMES[(T + H + D) % len(SCHEMES)]
    kw = dict(rot_dim=rot_dim, rot_off=rot_off, half=half)
    for inverse in (False, True):
        y = torch.full((T, H, D), float("nan"), dtype=x.dtype, device="cuda")
        mla.mla_rope_apply(pos, x, params=mla.rope_params(**sch), out=y, inverse=inverse, **kw)
        check(y, x, pos, sch, inverse=inverse, **kw)
    whole = torch.full((T, H, D + pad), 3.0, dtype=x.dtype, device="cuda")
    z = whole[:, :, :D]
    z.copy_(x)
    mla.mla_rope_apply(pos, z, params=mla.rope_params(**sch), inverse=True, **kw)
    assert torch.equal(z, y) and (whole[:, :, D:] == 3).all()  # the same bits in place, and nothing behind a head


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H,D,rot_off,rot_dim", [(2001, 17, 21, 3, 10), (3001, 40, 9, 1, 8), (700, 5, 401, 0, 6)])
def test_single_values_many_tokens(T, H, D, rot_off, rot_dim, dtype, half):
    """Rows without a 16-byte alignment where a thread walks several heads."""
    import mla_sparse_top_gb300 as mla
    x, pos = inputs(T, H, D, TYPES[dtype], pad=3, seed=H)
    scheme = SCHEMES[1]
    kw = dict(rot_dim=rot_dim, rot_off=rot_off, half=half)
    out = torch.full((T, H, D), float("nan"), dtype=x.dtype, device="cuda")
    mla.mla_rope_apply(pos, x, params=mla.rope_params(**scheme), out=out, **kw)
    check(out, x, pos, scheme, **kw)
    y = torch.full((T, H, D + 3), -7.0, dtype=x.dtype, device="cuda")
    y[:, :, :D] = x
    mla.mla_rope_apply(pos, y[:, :, :D], params=mla.rope_params(**scheme), **kw)
    assert torch.equal(y[:, :, :D], out) and (y[:, :, D:] == -7).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_two_tensors_keys_to_cache_rows(dtype):
    """Queries in place, keys into their rows of a cache; other rows stay, negative rows are skipped."""
    import mla_sparse_top_gb300 as mla
    T = 50
    q, pos = inputs(T, 64, 128, TYPES[dtype], seed=1)
    k, _ = inputs(T, 1, 128, TYPES[dtype], seed=2)
    cache = torch.full((300, 1, 128), 7.0, dtype=q.dtype, device="cuda")
    rows = torch.from_numpy(np.random.default_rng(0).permutation(300)[:T].astype(np.int64))
    rows[5], rows[6] = -1, -(2 ** 40)
    x = q.clone()
    sch = SCHEMES[3]
    mla.mla_rope_apply(pos, x, k, params=mla.rope_params(**sch), rot_dim=64, half=True, k_out=cache, k_rows=rows.cuda())
    assert mla.rope_device_status(clear=True) == 0
    check(x, q, pos, sch, rot_dim=64, rot_off=0, half=True)
    keep = rows >= 0
    check(cache[rows[keep].cuda()], k[keep.cuda()], pos[keep.cuda()], sch, rot_dim=64, rot_off=0, half=True)
    untouched = torch.ones(300, dtype=torch.bool)
    untouched[rows[keep]] = False
    assert (cache[untouched.cuda()] == 7).all()


def test_row_behind_the_cache_is_flagged():
    import mla_sparse_top_gb300 as mla
    k, pos = inputs(4, 1, 64, torch.bfloat16)
    cache = torch.zeros((11, 1, 64), dtype=k.dtype, device="cuda")
    view = cache[:10]
    rows = torch.tensor([3, 10, 2 ** 40, 9], device="cuda")
    mla.mla_rope_apply(pos, k.clone(), k, params=mla.rope_params(), rot_dim=64, k_out=view, k_rows=rows)
    assert mla.rope_device_status(clear=True) == mla.MLA_DEVICE_BAD_BLOCK
    assert mla.rope_device_status() == 0
    assert (cache[10] == 0).all() and (cache[[3, 9]] != 0).any(-1).all()


def test_heads_first_layout_and_broadcast_input():
    import mla_sparse_top_gb300 as mla
    x, pos = inputs(40, 6, 64, torch.bfloat16)
    hf = torch.empty((6, 40, 64), dtype=x.dtype, device="cuda")
    mla.mla_rope_apply(pos, x, params=mla.rope_params(), rot_dim=32, rot_off=32, out=hf.transpose(0, 1))
    check(hf.transpose(0, 1).contiguous(), x, pos, {}, rot_dim=32, rot_off=32, half=False)
    one = x[:, :1].expand(40, 6, 64)
    y = torch.empty_like(x)
    mla.mla_rope_apply(pos, one, params=mla.rope_params(), rot_dim=64, out=y)
    check(y, one.contiguous(), pos, {}, rot_dim=64, rot_off=0, half=False)


def test_inverse_is_the_gradient():
    """<R x, y> = <x, R^T y> in exact arithmetic on the fp32 outputs, and against differences: the map is linear, so
    (R(x + e) - R(x)) . y over a unit step e in one value is that value of R^T y."""
    import mla_sparse_top_gb300 as mla
    x, pos = inputs(6, 3, 48, torch.float32)
    y, _ = inputs(6, 3, 48, torch.float32, seed=9)
    par = mla.rope_params(**SCHEMES[3])

    def rot(t, inverse):
        o = torch.empty_like(t)
        mla.mla_rope_apply(pos, t, params=par, rot_dim=40, rot_off=4, half=True, inverse=inverse, out=o)
        return o.double()
    g = rot(y, True)
    lhs, rhs = (rot(x, False) * y.double()).sum(), (x.double() * g).sum()
    size = float((x.double().abs() * g.abs()).sum())
    assert abs(float(lhs - rhs)) <= 24 * U * 1.37 * 2 * size
    for at in [(0, 0, 4), (2, 1, 23), (5, 2, 43), (3, 0, 47)]:
        e = torch.zeros_like(x)
        e[at] = 1.0
        diff = (rot(e, False) * y.double()).sum()  # R(x + e) - R(x) = R(e)
        assert abs(float(diff - g[at])) <= 24 * U * 1.37 * float(y[at[0], at[1]].abs().max()) * 2


def test_graph_replay_and_no_tokens():
    import mla_sparse_top_gb300 as mla
    x, pos = inputs(20, 4, 64, torch.bfloat16)
    y = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_rope_apply(pos, x, params=mla.rope_params(), rot_dim=64, out=y)
    pos.add_(5)
    g.replay()
    torch.cuda.synchronize()
    check(y, x, pos, {}, rot_dim=64, rot_off=0, half=False)
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    mla.mla_rope_apply(pos[:0], e, params=mla.rope_params(), rot_dim=64)
    mla.mla_rope_table(pos[:0], torch.empty((0, 32), device="cuda"), torch.empty((0, 32), device="cuda"),
                       params=mla.rope_params())


def test_binding_refuses_what_it_cannot_pass_on():
    import mla_sparse_top_gb300 as mla
    x, pos = inputs(4, 2, 64, torch.bfloat16)
    par = mla.rope_params()
    for bad in (dict(positions=pos.long()), dict(q=x.double()), dict(q=x.transpose(1, 2)), dict(q=x.cpu()),
                dict(k=x.float()), dict(out=x[:3]), dict(k_rows=pos.long())):
        kw = dict(positions=pos, q=x, params=par, rot_dim=32)
        kw.update(bad)
        with pytest.raises(ValueError):
            mla.mla_rope_apply(**kw)
