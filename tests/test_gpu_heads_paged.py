"""Attention of new tokens over the pages on the GPU against the fp64 oracle (bounds in heads_util.py)."""
import numpy as np
import pytest
import torch

from heads_util import TYPES, cache, check_sequence, gather, normal, padded, page_table

pytestmark = pytest.mark.gpu


def make(act, *, S1=1, H=8, Hkv=2, D=128, Dv=128, dtype="bf16", layout="token", q_lens=None, pad=0, seed=0, W=None,
         scale=None, dead=float("nan")):
    gen = torch.Generator().manual_seed(seed + sum(act) + S1)
    dt, B = TYPES[dtype], len(act)
    table, used = page_table(gen, act, W)
    m = dict(act=act, S1=S1, H=H, Hkv=Hkv, D=D, Dv=Dv, dtype=dt, q_lens=q_lens, table_cpu=table,
             scale=D ** -0.5 if scale is None else scale, q=padded(gen, B * S1, H, D, dt, pad))
    for name, d in (("k", D), ("v", Dv)):
        x = m[name] = cache(used, Hkv, d, layout, dt, fill=dead)
        for b, a in enumerate(act):
            for p in range(min(-(-a // 128), table.shape[1])):
                n = min(128, a - 128 * p)
                x[table[b, p], :n] = normal(gen, (n, Hkv, d), dt)
    m["table"], m["act_gpu"] = table.cuda(), torch.tensor(act, dtype=torch.int32).cuda()
    m["lens_gpu"] = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32).cuda()
    return m


def run(m, lse=True, workspace=None):
    import mla_sparse_top_gb300 as mla
    T = m["q"].shape[0]
    out = torch.full((T, m["H"], m["Dv"]), float("nan"), dtype=m["dtype"], device="cuda")
    l = torch.full((T, m["H"]), float("nan"), device="cuda") if lse else None
    dims = mla.paged_dims(m["q"], m["k"], m["v"], m["table"], S1=m["S1"])
    if workspace is None:
        workspace = torch.full((mla.mla_paged_workspace_bytes(dims),), 255, dtype=torch.uint8, device="cuda")
    mla.mla_paged_attn_fwd(m["q"], m["k"], m["v"], m["table"], m["act_gpu"], out, l, workspace, q_lens=m["lens_gpu"],
                           softmax_scale=m["scale"], dims=dims)
    return out, l


def check(m, out, lse, status=0):
    import mla_sparse_top_gb300 as mla
    assert mla.heads_device_status(clear=True) == status
    S1 = m["S1"]
    for b, a in enumerate(m["act"]):
        n = S1 if m["q_lens"] is None else min(S1, max(0, m["q_lens"][b]))
        k, v = gather(m["k"], m["table_cpu"], b, max(0, a)), gather(m["v"], m["table_cpu"], b, max(0, a))
        rows = slice(b * S1, b * S1 + n)
        check_sequence(out[rows], lse[rows], m["q"][rows], k, v, m["scale"], True, f"sequence {b}")
        pad = slice(b * S1 + n, (b + 1) * S1)
        assert (out[pad] == 0).all() and torch.isneginf(lse[pad]).all()


CASES = [
    dict(act=[1]), dict(act=[0, 1, 2]), dict(act=[127, 128, 129, 63, 64, 65]), dict(act=[1000], H=16, D=64, Dv=64),
    dict(act=[500, 3, 2000], H=4, Hkv=4), dict(act=[700], H=7, Hkv=1, dtype="fp16"),
    dict(act=[300, 9000], H=40, Hkv=8, D=96, Dv=96, dtype="fp16"), dict(act=[260, 1], H=128, Hkv=1, D=192, Dv=128),
    dict(act=[100, 200], H=32, Hkv=1, D=64, Dv=128), dict(act=[129], H=10, Hkv=2, D=8, Dv=16, pad=8),
    dict(act=[513] * 40, H=3, Hkv=1, D=72, Dv=40), dict(act=[77, 1500], H=64, Hkv=4, D=128, Dv=64),
    dict(act=[40000], H=8, Hkv=1, D=64, Dv=64), dict(act=[20000, 50, 3000], H=4, Hkv=2),
    dict(act=[33, 900], H=20, Hkv=1, D=120, Dv=88, dtype="fp16"), dict(act=[2000], H=100, Hkv=2, D=128, Dv=128),
    dict(act=[64 * i for i in range(30)], H=2, Hkv=1, D=64, Dv=64),
]


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("case", CASES)
def test_single_tokens(case, layout):
    m = make(layout=layout, **case)
    check(m, *run(m))


@pytest.mark.parametrize("S1,act,kw", [
    (2, [1, 2, 3, 128, 129], {}), (5, [300, 131, 4, 2000], dict(H=10, Hkv=2, dtype="fp16")), (8, [700, 64], dict(H=8, Hkv=8)),
    (3, [400, 5], dict(H=64, Hkv=2, D=192)), (16, [129, 1000], dict(H=4, Hkv=1, D=64, Dv=64)), (33, [200, 33], dict(H=2, Hkv=1)),
    (64, [900], dict(H=4, Hkv=4)), (130, [131, 500], dict(H=3, Hkv=1, D=64, Dv=64)), (2, [300], dict(H=64, Hkv=1)),
    (4, [5000, 90], dict(H=16, Hkv=1, D=96, Dv=96, dtype="fp16"))])
def test_chains(S1, act, kw):
    m = make(act, S1=S1, layout="shared", **kw)
    check(m, *run(m))


def test_padded_batches():
    for S1, lens in ((1, [1, 0, 1, -3]), (5, [5, 0, 2, 9]), (20, [20, 1, 0, 7])):
        m = make([300, 40, 1000, 77], S1=S1, q_lens=lens, H=8, Hkv=2)
        check(m, *run(m))
    m = make([2, 1, 0, 5], S1=5, q_lens=[4, 4, 5, 5], H=8, Hkv=2)  # fewer keys than new tokens
    check(m, *run(m))


def test_scales_and_growing_scores():
    for scale in (0.0, -0.3, 3.0):
        m = make([700, 5], H=4, Hkv=1, D=64, Dv=64, scale=scale)
        check(m, *run(m))


def test_negative_lengths_count_as_none():
    m = make([100, 50], H=4, Hkv=2)
    m["act_gpu"][1] = -7
    m["act"] = [100, -7]
    check(m, *run(m))


def test_without_lse_and_repeated():
    m = make([3000, 77, 900], H=8, Hkv=2)
    a, l = run(m)
    b, _ = run(m, lse=False)
    c, l2 = run(m)
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(l, l2)


def test_batches_do_not_change_a_sequence():
    """A sequence's own keys alone decide what it gets, up to how they are shared out."""
    m = make([900, 4000, 33], H=8, Hkv=2, seed=9)
    check(m, *run(m))
    one = make([900], H=8, Hkv=2, seed=9)
    check(one, *run(one))


@pytest.mark.parametrize("S1,H", [(1, 8), (4, 8), (40, 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_reach_those_that_see_them(bad, S1, H):
    m = make([300, 200], S1=S1, H=H, Hkv=2, seed=2)
    clean = [x.clone() for x in run(m)]
    pos = 300 - (S1 + 1) // 2  # the chain's middle, or its only token
    m["v"][m["table_cpu"][0, pos // 128], pos % 128, 1, 5] = bad
    out, lse = run(m)
    first = max(0, pos - (300 - S1))
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[first:S1, H // 2:, 5] = True
    hit = hit.cuda()
    assert not torch.isfinite(out[hit]).any()
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse, clean[1])
    m["k"][m["table_cpu"][0, pos // 128], pos % 128, 1, 5] = float("nan")
    out, lse = run(m)
    rows = hit.any(-1)
    assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all()
    assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse[~rows], clean[1][~rows])


def test_bad_pages_and_a_short_table():
    import mla_sparse_top_gb300 as mla
    m = make([600, 300], H=8, Hkv=2, D=64, Dv=64)
    m["table"][0, 2] = 1 << 20
    m["table"][1, 0] = -1
    out, lse = run(m)
    assert mla.heads_device_status(clear=True) == mla.MLA_DEVICE_BAD_BLOCK
    for b, gone in ((0, 2), (1, 0)):
        a = m["act"][b]
        seen = np.ones(a, bool)
        seen[gone * 128:gone * 128 + 128] = False
        k, v = gather(m["k"], m["table_cpu"], b, a), gather(m["v"], m["table_cpu"], b, a)
        check_sequence(out[b:b + 1], lse[b:b + 1], m["q"][b:b + 1], k, v, m["scale"], True, f"sequence {b}", seen)
    m = make([500], H=4, Hkv=2, D=64, Dv=64, W=3)
    out, lse = run(m)
    assert mla.heads_device_status(clear=True) == mla.MLA_DEVICE_BAD_BLOCK
    seen = np.arange(500) < 384
    k, v = (torch.cat([gather(m[x], m["table_cpu"], 0, 384), torch.zeros((116, 2, 64), dtype=m["dtype"])]) for x in ("k", "v"))
    check_sequence(out, lse, m["q"], k, v, m["scale"], True, "short table", seen)


def test_wide_table_and_far_pages():
    """A table much wider than the lengths; pages whose offset passes 32 bits."""
    m = make([700, 300], H=8, Hkv=2, W=5000)
    check(m, *run(m))
    import mla_sparse_top_gb300 as mla
    blocks = 80000  # 80000 * 128 * 2 * 128 values: beyond 2^31 elements
    big = torch.empty((blocks, 128, 2, 128), dtype=torch.bfloat16, device="cuda")
    m = make([200], H=4, Hkv=2)
    far = torch.tensor([[blocks - 1, blocks - 3]], dtype=torch.int32)
    for i in range(2):
        big[far[0, i].item()] = m["k"][m["table_cpu"][0, i].item()]
    m["k"] = m["v"] = big
    m["table"], m["table_cpu"] = far.cuda(), far
    out, lse = run(m)
    assert mla.heads_device_status(clear=True) == 0
    k = torch.cat([big[blocks - 1].cpu(), big[blocks - 3].cpu()])[:200]
    check_sequence(out, lse, m["q"], k, k, m["scale"], True, "far pages")


def test_captured_and_replayed_on_new_lengths():
    import mla_sparse_top_gb300 as mla
    m = make([5000, 300, 64], H=8, Hkv=2, seed=4)
    dims = mla.paged_dims(m["q"], m["k"], m["v"], m["table"], S1=1)
    ws = torch.empty(mla.mla_paged_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    want = run(m)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_paged_attn_fwd(m["q"], m["k"], m["v"], m["table"], m["act_gpu"], out, lse, ws, softmax_scale=m["scale"], dims=dims)
    for act in ([5000, 300, 64], [4000, 0, 1], [128, 129, 2]):
        m["act"] = act
        m["act_gpu"].copy_(torch.tensor(act, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        check(m, out, lse)


def test_two_streams_with_a_workspace_each():
    ms = [make([6000, 40], H=8, Hkv=2, seed=i) for i in range(2)]
    want = [run(m) for m in ms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ms]
    got = []
    for _ in range(3):
        for m, s in zip(ms, streams):
            with torch.cuda.stream(s):
                got.append(run(m))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_a_wait_that_runs_out_is_reported_and_the_next_call_runs():
    """A bound far below the first load's latency: a launch that gives up reports it, and the next one does the whole
    job.  (One test of a barrier may suspend the warp for longer than a wait lasts: then the launch comes through.)"""
    import mla_sparse_top_gb300 as mla
    m = make([3000, 500], H=8, Hkv=2)
    want = run(m)
    assert mla.heads_device_status(clear=True) == 0
    mla.set_wait_limit_ns(1000)
    try:
        short = run(m)
        status = mla.heads_device_status(clear=True)
    finally:
        mla.set_wait_limit_ns(mla.DEFAULT_WAIT_LIMIT_NS)
    assert status in (0, mla.MLA_DEVICE_TIMEOUT)
    assert status != 0 or torch.equal(short[0], want[0])
    got = run(m)
    assert mla.heads_device_status(clear=True) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
