"""The page plan on the GPU against its oracle, integer for integer: padded
and packed rows, trees, lengths of zero, pages that end inside the new tokens,
lists that run out, bad ids, and two captured replays."""
import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu


def make(seed, B, S1, hi, new_hi, *, tree=False, spare=3, W=None, capacity=None):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, hi + 1, B)
    ctx[rng.random(B) < 0.2] = 0
    ctx[rng.random(B) < 0.2] //= 128
    new = rng.integers(0, new_hi + 1, B)
    have, need = -(-ctx // 128), -(-(ctx + new) // 128) - -(-ctx // 128)
    W = W or max(1, int((have + need).max()))
    num_blocks = int(have.sum() + need.sum()) + 50
    perm = rng.permutation(num_blocks).astype(np.int32)
    table = np.full((B, W), -7, dtype=np.int32)
    at = 0
    for b in range(B):
        n = min(W, have[b])
        table[b, :n] = perm[at:at + n]
        at += have[b]
    parents = None
    if tree:
        parents = (rng.random((B, S1)) * (np.arange(S1) + 1)).astype(np.int32) - 1
        parents[rng.random((B, S1)) < 0.05] = 2 ** 30  # outside: follows the context
    return dict(ctx=ctx.astype(np.int32), new=new.astype(np.int32), free=perm[at:at + max(0, int(need.sum()) + spare)],
                table=table, S1=S1, T=B * S1 if S1 else (capacity if capacity is not None else int(new.sum()) + 5),
                num_blocks=num_blocks, parents=parents)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(m, optional=True, stream=None, new="own"):
    import mla_sparse_top_gb300 as mla
    B, T, S1 = len(m["ctx"]), m["T"], m["S1"]
    i32 = dict(dtype=torch.int32, device="cuda")
    o = dict(act_seqs=torch.full((B,), -9, **i32), cache_index=torch.full((T,), -9, dtype=torch.int64, device="cuda"))
    if optional:
        o.update(positions=torch.full((T,), -9, **i32), seq_ids=torch.full((T,), -9, **i32),
                 cu_seqs=torch.full((B + 1,), -9, **i32), num_taken=torch.full((1,), -9, **i32))
        if S1:
            o["tree_mask"] = torch.full((T, -(-S1 // 64)), -9, dtype=torch.int64, device="cuda")
    table = dev(m["table"])
    mla.mla_page_plan(dev(m["ctx"]), dev(m["new"]) if new == "own" else None, dev(m["free"].astype(np.int32)), table,
                      S1=S1, num_blocks=m["num_blocks"], parents=dev(m["parents"]), stream=stream, **o)
    status = mla.page_device_status(clear=True, stream=stream)
    return {k: v.cpu().numpy() for k, v in o.items()} | {"block_table": table.cpu().numpy(), "status": status}


def check(m, got, new="own"):
    want = step.page_plan(m["ctx"], m["new"] if new == "own" else None, m["free"], m["table"], S1=m["S1"], T=m["T"],
                          num_blocks=m["num_blocks"], parents=m["parents"])
    for k, v in got.items():
        if k == "tree_mask":
            words = [[(bits >> 64 * w) & (2 ** 64 - 1) for w in range(v.shape[1])] for bits in want[k]]
            np.testing.assert_array_equal(v.view(np.uint64), np.array(words, dtype=np.uint64).reshape(v.shape), k)
        else:
            np.testing.assert_array_equal(v, want[k], k)
    return want


@pytest.mark.parametrize("B,S1,hi,tree", [(1, 1, 0, False), (1, 1, 500, True), (64, 8, 8192, True), (7, 64, 300, True),
                                          (5, 65, 1000, True), (3, 300, 5000, True), (300, 3, 2000, False),
                                          (1000, 5, 700, True), (2, 1000, 100, False), (257, 1, 128, False)])
def test_padded_rows(B, S1, hi, tree):
    m = make(B + S1, B, S1, hi, S1 + 1, tree=tree)  # some new lengths above S1: they count as S1
    assert check(m, run(m))["status"] == 0


@pytest.mark.parametrize("B,hi,new_hi", [(1, 0, 1), (1, 300, 5000), (37, 65, 4096), (256, 500, 3), (1000, 1000, 40),
                                         (600, 0, 0), (513, 9000, 9)])
def test_packed_rows(B, hi, new_hi):
    m = make(B + hi, B, 0, hi, new_hi)
    assert check(m, run(m))["status"] == 0


def test_required_outputs_alone_and_default_lengths():
    m = make(3, 20, 4, 900, 4)
    check(m, run(m, optional=False))
    m["free"] = np.arange(m["num_blocks"], dtype=np.int32)
    check(m, run(m, new=None), new=None)


def test_negative_lengths_count_as_zero():
    m = make(4, 20, 4, 900, 4)
    m["ctx"][3], m["new"][4] = -5, -2 ** 31
    check(m, run(m))


@pytest.mark.parametrize("S1", [0, 6])
def test_free_list_runs_out(S1):
    m = make(5, 40, S1, 300, 6 if S1 else 700, spare=-4)
    assert check(m, run(m))["status"] == step.NO_PAGE


def test_no_free_blocks_at_all():
    m = make(6, 3, 4, 100, 4)
    m["ctx"][:] = [0, 10, 126]
    m["table"][:, 0] = [-1, 1, 2]
    m["new"][:] = 4
    m["free"] = m["free"][:0]
    assert check(m, run(m))["status"] == step.NO_PAGE


@pytest.mark.parametrize("S1", [0, 300])
def test_table_too_narrow(S1):
    m = make(7, 9, S1, 600, 300, W=3)
    assert check(m, run(m))["status"] == step.NO_PAGE


def test_packed_capacity_too_small():
    m = make(8, 30, 0, 600, 300, capacity=1500)
    assert int(m["new"].sum()) > 1500
    assert check(m, run(m))["status"] == step.NO_PAGE


@pytest.mark.parametrize("bad", [-3, 10 ** 6])
def test_bad_ids_are_flagged_not_followed(bad):
    m = make(9, 12, 4, 900, 4)
    m["ctx"][5], m["new"][5] = 130, 3
    m["table"][5, 1] = bad
    assert check(m, run(m))["status"] == step.BAD_BLOCK


def test_no_sequences_is_a_no_op():
    m = dict(ctx=np.zeros(0, np.int32), new=np.zeros(0, np.int32), free=np.zeros(0, np.int32),
             table=np.zeros((0, 1), np.int32), S1=4, T=0, num_blocks=1, parents=None)
    got = run(m, optional=False)
    assert got["status"] == 0 and got["cache_index"].size == 0


def test_largest_lengths_do_not_wrap():
    m = dict(ctx=np.array([2 ** 31 - 2, 2 ** 31 - 1], np.int32), new=np.array([4, 4], np.int32),
             free=np.arange(4, dtype=np.int32), table=np.full((2, 2), 1, np.int32), S1=4, T=8, num_blocks=4,
             parents=None)
    got = run(m)
    assert got["act_seqs"].tolist() == [2 ** 31 - 1] * 2 and got["status"] == step.NO_PAGE
    assert (got["cache_index"] == -1).all() and (got["positions"] >= 0).all()
    assert got["block_table"].tolist() == m["table"].tolist()


def test_same_plan_from_a_graph_and_on_another_stream():
    import mla_sparse_top_gb300 as mla
    m = make(11, 50, 8, 3000, 8, tree=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        check(m, run(m, stream=s))
    ctx, new, free, par = dev(m["ctx"]), dev(m["new"]), dev(m["free"]), dev(m["parents"])
    table = dev(m["table"])
    act, idx = torch.zeros(50, dtype=torch.int32, device="cuda"), torch.zeros(400, dtype=torch.int64, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_page_plan(ctx, new, free, table, act, idx, S1=8, num_blocks=m["num_blocks"], parents=par)
    m2 = make(12, 50, 8, 2500, 8, tree=True)  # other lengths through the same graph
    for mm in (m, m2):
        mm["num_blocks"] = m["num_blocks"]
        W, F = table.shape[1], free.numel()
        wide = np.full((50, W), -1, np.int32)
        w = min(W, mm["table"].shape[1])
        wide[:, :w] = mm["table"][:, :w]
        mm["table"], mm["free"] = wide, np.resize(mm["free"], F).astype(np.int32)
        ctx.copy_(dev(mm["ctx"])), new.copy_(dev(mm["new"])), free.copy_(dev(mm["free"])), par.copy_(dev(mm["parents"]))
        table.copy_(dev(mm["table"]))
        g.replay()
        torch.cuda.synchronize()
        want = step.page_plan(mm["ctx"], mm["new"], mm["free"], mm["table"], S1=8, T=400, num_blocks=m["num_blocks"],
                              parents=mm["parents"])
        np.testing.assert_array_equal(idx.cpu().numpy(), want["cache_index"])
        np.testing.assert_array_equal(table.cpu().numpy(), want["block_table"])
    mla.page_device_status(clear=True)
