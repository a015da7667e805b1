"""Attention over whole prompts on the GPU against the fp64 oracle (bounds in heads_util.py)."""
import numpy as np
import pytest
import torch

from heads_util import TYPES, cache, check_gpu, check_sequence, gather, normal, np64, padded, page_table

pytestmark = pytest.mark.gpu


def make(lens, *, ctx=None, H=4, Hkv=2, D=64, Dv=64, dtype="bf16", paged=False, causal=True, layout="token", pad=0,
         spare=5, begin=0, kv_lens=None, seed=0, scale=None, W=None, dead=float("nan")):
    """A call's tensors; what must not matter (rows behind a sequence, unused pages) holds `dead`."""
    gen = torch.Generator().manual_seed(seed + sum(lens))
    dt = TYPES[dtype]
    B, T = len(lens), begin + sum(lens) + spare
    m = dict(lens=lens, H=H, Hkv=Hkv, D=D, Dv=Dv, causal=causal, begin=begin, scale=D ** -0.5 if scale is None else scale,
             paged=paged, dtype=dt)
    m["q"] = padded(gen, T, H, D, dt, pad)
    m["cu_q"] = (torch.tensor([0] + lens).cumsum(0) + begin).to(torch.int32).cuda()
    m["cu_k"] = m["table"] = m["act"] = None
    if paged:
        act = [c + n for c, n in zip(ctx or [0] * B, lens)]
        table, used = page_table(gen, act, W)
        m["act_list"] = act
        m["k"], m["v"] = cache(used, Hkv, D, layout, dt, fill=dead), cache(used, Hkv, Dv, layout, dt, fill=dead)
        for b, a in enumerate(act):
            for p in range(-(-a // 128)):
                if p < table.shape[1]:
                    n = min(128, a - 128 * p)
                    m["k"][table[b, p], :n] = normal(gen, (n, Hkv, D), dt)
                    m["v"][table[b, p], :n] = normal(gen, (n, Hkv, Dv), dt)
        m["table_cpu"] = table
        m["table"], m["act"] = table.cuda(), torch.tensor(act, dtype=torch.int32).cuda()
    else:
        kl = lens if kv_lens is None else kv_lens
        m["kl"] = kl
        Tk = begin + sum(kl) + spare
        m["k"], m["v"] = padded(gen, Tk, Hkv, D, dt, pad), padded(gen, Tk, Hkv, Dv, dt, pad)
        m["k"][begin + sum(kl):] = dead
        m["v"][begin + sum(kl):] = dead
        if kv_lens is not None:
            m["cu_k"] = (torch.tensor([0] + kl).cumsum(0) + begin).to(torch.int32).cuda()
    return m


def run(m, lse=True, workspace=None, out=None, **kw):
    import mla_sparse_top_gb300 as mla
    T = m["q"].shape[0]
    if out is None:
        out = torch.full((T, m["H"], m["Dv"]), 7.0, dtype=m["dtype"], device="cuda")
    l = torch.full((T, m["H"]), 7.0, device="cuda") if lse else None
    dims = mla.prompt_dims(m["q"], m["k"], m["v"], m["cu_q"], block_table=m["table"], causal=m["causal"])
    if workspace is None:
        workspace = torch.full((mla.mla_prompt_workspace_bytes(dims),), 255, dtype=torch.uint8, device="cuda")
    mla.mla_prompt_attn_fwd(m["q"], m["k"], m["v"], m["cu_q"], out, l, workspace, cu_k=m["cu_k"], block_table=m["table"],
                            act_seqs=m["act"], softmax_scale=m["scale"], dims=dims, **kw)
    return out, l


def keys_of(m, b):
    if m["paged"]:
        a = m["act_list"][b]
        return gather(m["k"], m["table_cpu"], b, a), gather(m["v"], m["table_cpu"], b, a)
    k0 = m["begin"] + sum(m["kl"][:b])
    return m["k"][k0:k0 + m["kl"][b]], m["v"][k0:k0 + m["kl"][b]]


def check(m, out, lse, status=0):
    import mla_sparse_top_gb300 as mla
    assert mla.heads_device_status(clear=True) == status
    at = m["begin"]
    assert (out[:at] == 7).all() and (lse[:at] == 7).all()
    for b, n in enumerate(m["lens"]):
        k, v = keys_of(m, b)
        check_sequence(out[at:at + n], lse[at:at + n], m["q"][at:at + n], k, v, m["scale"], m["causal"], f"sequence {b}")
        at += n
    assert (out[at:] == 7).all() and (lse[at:] == 7).all()  # rows behind the last sequence


CASES = [
    dict(lens=[1]), dict(lens=[1, 1, 1], H=8, Hkv=8), dict(lens=[0, 0]), dict(lens=[5, 0, 130, 0]),
    dict(lens=[127, 128, 129], H=6, Hkv=2, D=128, Dv=128), dict(lens=[300], H=16, Hkv=4),
    dict(lens=[257, 31], H=7, Hkv=1, D=96, Dv=80, dtype="fp16"), dict(lens=[600, 3], H=2, Hkv=2, D=192, Dv=128),
    dict(lens=[255, 256, 257], H=1, Hkv=1, D=128, Dv=128), dict(lens=[33, 1000], H=12, Hkv=4, D=8, Dv=8),
    dict(lens=[200], H=128, Hkv=1, D=64, Dv=64), dict(lens=[50, 70], H=48, Hkv=2, D=40, Dv=120, dtype="fp16"),
    dict(lens=[129, 64], H=9, Hkv=3, D=72, Dv=104, pad=8), dict(lens=[400, 20], causal=False, H=5, Hkv=5, D=128, Dv=64),
    dict(lens=[90, 300], begin=17, spare=130, H=4, Hkv=1, D=128, Dv=128),
    dict(lens=[700], H=3, Hkv=3, D=184, Dv=24, dtype="fp16"), dict(lens=[1500], H=2, Hkv=1, D=128, Dv=128, dtype="fp16"),
    dict(lens=list(range(1, 60)), H=4, Hkv=2),
]


@pytest.mark.parametrize("case", CASES)
def test_packed(case):
    m = make(**case)
    check(m, *run(m))


@pytest.mark.parametrize("lens,kv,causal", [([100], [300], True), ([100, 7], [40, 7], True), ([3, 200, 60], [0, 129, 1000], False),
                                            ([300, 300], [0, 5], True)])
def test_keys_of_other_lengths(lens, kv, causal):
    """Queries at the end of longer keys; fewer keys than queries leave the first ones nothing to see."""
    m = make(lens, kv_lens=kv, causal=causal, H=4, Hkv=2, D=128, Dv=128)
    check(m, *run(m))


@pytest.mark.parametrize("layout", ["token", "head", "shared"])
@pytest.mark.parametrize("lens,ctx,kw", [
    ([1, 2], [0, 5000], dict(H=8, Hkv=1, D=128, Dv=128)), ([64, 1, 300], [700, 0, 129], dict(H=4, Hkv=2, D=128, Dv=128)),
    ([17], [10000], dict(H=14, Hkv=2, D=64, Dv=64, dtype="fp16")), ([100, 0, 30], [28, 9, 0], dict(H=3, Hkv=3, D=192, Dv=128)),
    ([260], [1], dict(H=2, Hkv=2, D=80, Dv=80, causal=False))])
def test_paged(lens, ctx, kw, layout):
    m = make(lens, ctx=ctx, paged=True, layout=layout, **kw)
    check(m, *run(m))


def test_long_context_is_shared_out():
    """Few rows over many keys: the parts that several SMs made are joined."""
    m = make([3, 40], ctx=[30000, 7000], paged=True, H=8, Hkv=2, D=128, Dv=128, seed=3)
    check(m, *run(m))
    m = make([5], kv_lens=[20000], H=4, Hkv=4, D=64, Dv=64, causal=False)
    check(m, *run(m))


def test_scales():
    for scale in (0.0, -0.3, 2.0):
        m = make([150], H=2, Hkv=1, D=64, Dv=64, scale=scale)
        check(m, *run(m))


def test_large_scores_move_the_maximum():
    """Scores that grow along the keys: the running maximum moves in every tile."""
    m = make([900], H=2, Hkv=1, D=64, Dv=64, scale=1.0)
    m["k"].mul_((torch.arange(m["k"].shape[0], device="cuda")[:, None, None] / 100).to(m["k"].dtype))
    m["k"][900:] = 0
    check(m, *run(m))


def test_without_lse_and_repeated():
    m = make([300, 77], H=8, Hkv=2, D=128, Dv=128)
    a, l = run(m)
    b, _ = run(m, lse=False)
    c, l2 = run(m)
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(l, l2)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_non_finite_rows_reach_those_that_see_them(bad, where):
    m = make([70, 300, 200], H=4, Hkv=2, D=128, Dv=128, seed=5)
    m["k"][370:] = 0
    m["v"][370:] = 0
    clean = [x.clone() for x in run(m)]
    pos = 200  # of sequence 1
    m[where][70 + pos, 1, 3] = bad
    out, lse = run(m)
    reached = torch.zeros(out.shape[:2], dtype=torch.bool)
    reached[70 + pos:370, 2:] = True
    same = ~reached.cuda()
    assert torch.equal(out[same], clean[0][same]) and torch.equal(lse[same], clean[1][same])
    hit = out[reached.cuda()]
    if where == "v":
        assert not torch.isfinite(hit[:, 3]).any()
        others = [d for d in range(128) if d != 3]
        assert torch.equal(hit[:, others], clean[0][reached.cuda()][:, others])
        assert torch.equal(lse, clean[1])
    elif bad != bad:
        assert torch.isnan(hit).all() and torch.isnan(lse[reached.cuda()]).all()


def test_non_finite_queries_stay_with_their_rows():
    m = make([300], H=4, Hkv=2, D=64, Dv=64)
    clean = [x.clone() for x in run(m)]
    m["q"][100, 1] = float("nan")
    out, lse = run(m)
    same = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    same[100, 1] = False
    assert torch.equal(out[same], clean[0][same]) and torch.isnan(out[100, 1]).all() and torch.isnan(lse[100, 1])


def test_keys_that_all_score_minus_infinity():
    m = make([40], H=2, Hkv=1, D=8, Dv=8)
    m["q"].fill_(1.0)
    m["k"].fill_(-float("inf"))
    out, lse = run(m)
    assert (out[:40] == 0).all() and torch.isneginf(lse[:40]).all()


def test_bad_pages_and_a_short_table():
    import mla_sparse_top_gb300 as mla
    m = make([50, 60], ctx=[300, 200], paged=True, H=4, Hkv=2, D=64, Dv=64)
    m["table"][0, 1] = 99999
    m["table"][1, 0] = -1
    out, lse = run(m)
    assert mla.heads_device_status(clear=True) == mla.MLA_DEVICE_BAD_BLOCK
    for b, at, gone in ((0, 0, 1), (1, 50, 0)):
        n, a = m["lens"][b], m["act_list"][b]
        seen = np.ones(a, bool)
        seen[gone * 128:gone * 128 + 128] = False
        k, v = keys_of(m, b)
        check_sequence(out[at:at + n], lse[at:at + n], m["q"][at:at + n], k, v, m["scale"], True, f"sequence {b}", seen)
    m = make([20], ctx=[400], paged=True, H=4, Hkv=2, D=64, Dv=64, W=2)
    out, lse = run(m)
    assert mla.heads_device_status(clear=True) == mla.MLA_DEVICE_BAD_BLOCK
    seen = np.arange(420) < 256
    k, v = (torch.cat([gather(m[x], m["table_cpu"], 0, 256), torch.zeros((164, 2, 64), dtype=m["dtype"])]) for x in ("k", "v"))
    check_sequence(out[:20], lse[:20], m["q"][:20], k, v, m["scale"], True, "short table", seen)


def test_bad_offsets_are_clamped():
    import mla_sparse_top_gb300 as mla
    m = make([40, 50], H=2, Hkv=1, D=64, Dv=64, spare=0)
    for cu in ([-5, 40, 90], [0, 40, 1000], [0, 60, 40]):
        m["cu_q"] = torch.tensor(cu, dtype=torch.int32).cuda()
        out, lse = run(m)
        assert mla.heads_device_status(clear=True) == mla.MLA_DEVICE_BAD_LENGTH
        n = min(cu[1], 90)
        check_sequence(out[:n], lse[:n], m["q"][:n], m["k"][:n], m["v"][:n], m["scale"], True, f"{cu}")


def test_views_of_one_fused_tensor():
    """Queries, keys and values as one projection leaves them."""
    import mla_sparse_top_gb300 as mla
    T, H, Hkv, D = 333, 6, 2, 64
    x = normal(torch.Generator().manual_seed(1), (T, (H + 2 * Hkv) * D), torch.bfloat16)
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split((H * D, Hkv * D, Hkv * D), 1))
    m = dict(q=q, k=k, v=v, cu_q=torch.tensor([0, 100, T], dtype=torch.int32).cuda(), cu_k=None, table=None, act=None, H=H,
             Hkv=Hkv, D=D, Dv=D, causal=True, scale=0.1, dtype=x.dtype, lens=[100, 233], kl=[100, 233], begin=0, paged=False)
    check(m, *run(m))
    assert mla.heads_device_status(clear=True) == 0


def test_other_stream_and_captured():
    m = make([200, 90], ctx=[0, 1000], paged=True, H=8, Hkv=2, D=128, Dv=128)
    want = run(m)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(m)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    import mla_sparse_top_gb300 as mla
    dims = mla.prompt_dims(m["q"], m["k"], m["v"], m["cu_q"], block_table=m["table"])
    ws = torch.empty(mla.mla_prompt_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_prompt_attn_fwd(m["q"], m["k"], m["v"], m["cu_q"], out, lse, ws, block_table=m["table"], act_seqs=m["act"],
                                softmax_scale=m["scale"], dims=dims)
    for _ in range(3):
        out.fill_(7.0), lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # new lengths, the same graph
    m["act"].copy_(torch.tensor([200, 700], dtype=torch.int32))
    m["act_list"] = [200, 700]
    out.fill_(7.0), lse.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    check(m, out, lse)
    assert np.isfinite(np64(out)).all()


# Calls with rows enough for pairs of SMs (512 rows at a time, at least 4096 of a key head for each sequence, two rounds in all), or nearly
LARGE = [
    dict(lens=[1300], H=128, Hkv=128, D=192, Dv=128, pad=8), dict(lens=[2049], H=80, Hkv=2, D=128, Dv=128, spare=40, begin=3),
    dict(lens=[1025, 1030, 2000], H=48, Hkv=16, D=96, Dv=80, dtype="fp16"), dict(lens=[5, 1500, 0, 1200], H=128, Hkv=4, D=64, Dv=72),
    dict(lens=[1281], H=128, Hkv=1, D=64, Dv=128, causal=False), dict(lens=[700, 900], ctx=[3000, 129], H=100, Hkv=4, D=128, Dv=128, paged=True, layout="head"),
    dict(lens=[1400], ctx=[77], H=112, Hkv=16, D=192, Dv=104, paged=True, layout="shared", dtype="fp16"),
    dict(lens=[4100], H=48, Hkv=48, D=192, Dv=128, spare=3), dict(lens=[1400, 1500, 1400], H=48, Hkv=16, D=96, Dv=80, dtype="fp16"),
    dict(lens=[60, 200], ctx=[40000, 9000], H=8, Hkv=2, D=128, Dv=128, paged=True), dict(lens=[33], ctx=[20000], H=6, Hkv=1, D=64, Dv=64, paged=True),
]


@pytest.mark.parametrize("case", LARGE)
def test_many_rows(case):
    import mla_sparse_top_gb300 as mla
    m = make(**case)
    out, lse = run(m)
    assert mla.heads_device_status(clear=True) == 0
    at = m["begin"]
    assert (out[:at] == 7).all() and (lse[:at] == 7).all()
    for b, n in enumerate(m["lens"]):
        k, v = keys_of(m, b)
        check_gpu(out[at:at + n], lse[at:at + n], m["q"][at:at + n], k.cuda(), v.cuda(), m["scale"], m["causal"], f"sequence {b}")
        at += n
    assert (out[at:] == 7).all() and (lse[at:] == 7).all()
    again, lse2 = run(m)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("rise", [1.0, -1.0, 0.0])
def test_many_rows_with_scores_that_grow(rise):
    """Maxima that move with every tile, by far more than weights may grow, and rows that score -inf at first."""
    import mla_sparse_top_gb300 as mla
    m = make([1400], H=112, Hkv=2, D=64, Dv=128, seed=3)
    n = 1400
    m["q"][:n] = m["q"][:n].abs()  # so that a key's scores have its sign
    steps = (torch.arange(n, device="cuda") // 100).float()
    m["k"][:n] = (m["k"][:n].float() * 0.1 + (rise * steps)[:, None, None]).to(m["dtype"])
    if rise == 0:
        m["k"][:300] = -float("inf")  # three tiles, the first rows see nothing else
    out, lse = run(m)
    assert mla.heads_device_status(clear=True) == 0
    if rise == 0:
        assert (out[:300] == 0).all() and torch.isneginf(lse[:300]).all()
        live = slice(300, n)  # their softmax is that over the finite keys
        check_gpu(out[live], lse[live], m["q"][live], m["k"][live], m["v"][live], m["scale"], True, "behind -inf")
    else:
        check_gpu(out[:n], lse[:n], m["q"][:n], m["k"][:n], m["v"][:n], m["scale"], True, f"rise {rise}")


def test_many_rows_with_values_that_are_not_finite():
    """A value in the half of the columns that the other SM of the pair holds reaches both SMs' rows, and no others."""
    m = make([1400], H=112, Hkv=2, D=128, Dv=128)
    m["k"][1400:] = 0
    m["v"][1400:] = 0
    clean = [x.clone() for x in run(m)]
    for col in (3, 100):
        m["v"][900, 1, col] = float("nan")
    out, lse = run(m)
    assert torch.equal(lse, clean[1]) and torch.equal(out[:, :56], clean[0][:, :56]) and torch.equal(out[:900], clean[0][:900])
    hit = out[900:1400, 56:]
    assert not torch.isfinite(hit[..., [3, 100]]).any()
    rest = [d for d in range(128) if d not in (3, 100)]
    assert torch.equal(hit[..., rest], clean[0][900:1400, 56:][..., rest])


@pytest.mark.parametrize("case", [dict(lens=[1400, 300], H=112, Hkv=2, D=128, Dv=128), dict(lens=[900], H=4, Hkv=2),
                                  dict(lens=[100, 40], ctx=[30000, 9000], H=16, Hkv=2, D=128, Dv=128, paged=True)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_runs(case):
    """A bound far below what a whole call waits: a launch that gives up reports it, and the next one does the whole job.

    The bound is looked at between tests of a barrier, and one test may suspend the warp for longer than the waits of
    a small call last: that one may come through, with its results whole."""
    import mla_sparse_top_gb300 as mla
    m = make(**case)
    want = run(m)
    assert mla.heads_device_status(clear=True) == 0
    mla.set_wait_limit_ns(1000)
    try:
        short = run(m)
        status = mla.heads_device_status(clear=True)
    finally:
        mla.set_wait_limit_ns(mla.DEFAULT_WAIT_LIMIT_NS)
    assert status == mla.MLA_DEVICE_TIMEOUT or (status == 0 and m["q"].shape[0] < 1000)
    assert status != 0 or torch.equal(short[0], want[0])
    got = run(m)
    assert mla.heads_device_status(clear=True) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
