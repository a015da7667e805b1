"""Dense attention of drafted tokens on the GPU against the fp64 oracle.

Bound of one output, with u = 2^-24 and h = 2^-8 (half a step of bf16,
relative): every softmax weight is rounded to bf16 once, which moves the
output by at most h sum_p p |v_p|; the output's own rounding by h |o|.  A score
is an fp32 sum of 576 exact products (error at most 576 u times the sum Z of
their magnitudes times |scale|, plus 2 u |z| from the scale), exp2 and the
running sums over L keys add (L + 16) u; an error d of all scores moves the
weights by 2 d relative.  lse moves by d, the sums' error and its own rounding."""
import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8


def parents_of(rng, B, S1):
    return (rng.random((B, S1)) * (np.arange(S1) + 1)).astype(np.int64) - 1


def masks_of(parents):
    out = []
    for row in parents:
        up = []
        for i, par in enumerate(row):
            up.append((up[par] if par >= 0 else 0) | 1 << i)
        out += up
    return out


def make(seed, act, S1, n_q, *, int8=False, tree=True, lens=None, poison=True, scale=None, spare=2, W=None):
    rng = np.random.default_rng(seed)
    B = len(act)
    blocks = [-(-max(0, a) // 128) for a in act]
    nb = sum(blocks) + spare
    table = np.full((B, W or max(1, max(blocks))), -1, np.int32)
    perm = rng.permutation(nb)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    g = torch.Generator().manual_seed(seed)
    rows = nb * 128
    live = np.zeros(rows, bool)
    for b in range(B):
        p = np.arange(max(0, act[b]))
        live[table[b, p // 128] * 128 + p % 128] = True
    dead = torch.from_numpy(~live)
    m = dict(S1=S1, act=np.array(act, np.int32), table=table, lens=None if lens is None else np.array(lens, np.int32),
             masks=masks_of(parents_of(rng, B, S1)) if tree else None,
             q_nope=torch.randn((B * S1, n_q, 512), generator=g).bfloat16(),
             q_rope=torch.randn((B * S1, n_q, 64), generator=g).bfloat16(),
             kv_rope=torch.randn((rows, 64), generator=g).bfloat16(), scales=None,
             scale=576 ** -0.5 if scale is None else scale)
    if int8:
        m["kv_nope"] = torch.randint(-128, 128, (rows, 512), generator=g).to(torch.int8)
        m["scales"] = (torch.rand((rows, 4), generator=g) + 0.5) / 64
    else:
        m["kv_nope"] = torch.randn((rows, 512), generator=g).bfloat16()
    if poison:  # what no token may see
        m["kv_rope"][dead] = float("nan")
        if int8:
            m["scales"][dead] = float("nan")
        else:
            m["kv_nope"][dead] = float("inf")
    return m


def words_of(masks, S1):
    n = -(-S1 // 64)
    w = np.array([[(x >> 64 * k) & (2 ** 64 - 1) for k in range(n)] for x in masks], dtype=np.uint64)
    return torch.from_numpy(w.view(np.int64)).cuda()


def upload(m):
    d = {k: m[k].cuda() for k in ("q_nope", "q_rope", "kv_nope", "kv_rope")}
    d["kv_scales"] = None if m["scales"] is None else m["scales"].cuda()
    d["block_table"] = torch.from_numpy(m["table"]).cuda()
    d["act_seqs"] = torch.from_numpy(m["act"]).cuda()
    d["tree_lens"] = None if m["lens"] is None else torch.from_numpy(m["lens"]).cuda()
    d["tree_mask"] = None if m["masks"] is None else words_of(m["masks"], m["S1"])
    return d


def launch(m, d, out, lse, ws=None, stream=None):
    import mla_sparse_top_gb300 as mla
    dims = mla.tree_dims(d["q_nope"], d["kv_nope"], d["block_table"], S1=m["S1"])
    if ws is None:
        ws = torch.full((mla.mla_tree_workspace_bytes(dims),), 0xFF, dtype=torch.uint8, device="cuda")
    mla.mla_tree_attn_fwd(d["q_nope"], d["q_rope"], d["kv_nope"], d["kv_rope"], d["kv_scales"], d["block_table"],
                          d["act_seqs"], out, lse, ws, tree_lens=d["tree_lens"], tree_mask=d["tree_mask"],
                          softmax_scale=m["scale"], dims=dims, stream=stream)
    return ws


def run(m, with_lse=True):
    import mla_sparse_top_gb300 as mla
    d = upload(m)
    out = torch.full_like(d["q_nope"], float("nan"))
    lse = torch.full(out.shape[:2], float("nan"), device="cuda") if with_lse else None
    ws = launch(m, d, out, lse)
    status = mla.tree_device_status(clear=True)
    again = torch.full_like(out, float("nan"))
    launch(m, d, again, None, ws)
    assert mla.tree_device_status(clear=True) == status
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits, and no need of lse
    return out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy(), status


def latent_of(m):
    if m["scales"] is None:
        return m["kv_nope"].double().numpy()
    return (m["kv_nope"].float() * m["scales"].repeat_interleave(128, 1)).bfloat16().double().numpy()


def check(m, got=None, tokens=None):
    out, lse, status = run(m) if got is None else got
    qn, qr = m["q_nope"].double().numpy(), m["q_rope"].double().numpy()
    lat, rope = latent_of(m), m["kv_rope"].double().numpy()
    o, e, mag = step.tree_attention(qn, qr, lat, rope, m["table"], m["act"], m["lens"], m["masks"], m["S1"], m["scale"])
    L = int(max(0, m["act"].max()))
    # sum of the magnitudes of a score's products, over all keys and rows
    keys = np.abs(np.nan_to_num(np.concatenate([lat, rope], 1), posinf=0, neginf=0))
    top = float(np.linalg.norm(keys, axis=1).max() * np.linalg.norm(np.concatenate([qn, qr], -1), axis=-1).max())
    d = abs(m["scale"]) * top * 578 * U + (L + 16) * U
    bound = (HALF + 2 * d) * mag * (1 + 2 * d) + HALF * np.abs(o) * 1.01 + 1e-30
    err = np.abs(out - o)
    assert (err <= bound).all(), f"out: worst {np.nanmax(err / bound)}, {(~(err <= bound)).sum()} of {err.size}"
    inf = np.isneginf(e)
    assert (np.isneginf(lse) == inf).all() and (out[inf] == 0).all()
    el = np.abs(lse[~inf] - e[~inf])
    assert (el <= d + 4 * U * (1 + np.abs(e[~inf]))).all(), f"lse: worst {el.max()} of {d}"
    return status


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("act", [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 511, 513, 1000])
def test_single_token_every_length(act, int8):
    m = make(act, [act], 1, 16, int8=int8, tree=False)
    assert check(m) == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("S1,n_q,act", [
    (1, 128, [700, 0, 1, 1500]), (2, 128, [2, 300, 129]), (8, 128, [900, 8, 257, 130]), (8, 16, [1000]),
    (3, 5, [400, 3, 70]), (17, 100, [500, 18]), (64, 16, [64, 700]), (65, 3, [300, 129]), (130, 1, [130, 131, 400]),
    (130, 7, [600]), (40, 128, [200])])
@pytest.mark.parametrize("tree", [False, True])
def test_drafts(S1, n_q, act, tree, int8):
    assert check(make(S1 * n_q, act, S1, n_q, int8=int8, tree=tree)) == 0


@pytest.mark.parametrize("int8", [False, True])
def test_drafts_of_unequal_size_and_padding(int8):
    m = make(1, [300, 5, 700, 260, 0, 9, 129], 9, 64, int8=int8, lens=[9, 3, 0, 1, 0, 20, -4])
    out, lse, status = run(m)
    assert check(m, (out, lse, status)) == 0
    pad = [b * 9 + s for b, n in enumerate([9, 3, 0, 1, 0, 9, 0]) for s in range(n, 9)]
    assert (out[pad] == 0).all() and np.isneginf(lse[pad]).all()


@pytest.mark.parametrize("int8", [False, True])
def test_long_contexts_cut_between_clusters(int8):
    assert check(make(2, [9000], 2, 128, int8=int8)) == 0
    assert check(make(3, [9000, 20, 4000], 5, 70, int8=int8)) == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("act,S1,n_q", [([20000], 1, 128), ([20000], 1, 1), ([300], 1, 100), ([6000, 0, 130, 5000], 3, 40),
                                        ([1000] * 8, 3, 96), ([40000], 2, 65)])
def test_tables_wider_than_the_lengths(act, S1, n_q, int8):
    """Room for more teams than there are tiles; row blocks with a part from almost every team."""
    assert check(make(31, act, S1, n_q, int8=int8, W=700)) == 0


def test_many_sequences():
    rng = np.random.default_rng(4)
    act = rng.integers(0, 400, 700).tolist()
    assert check(make(4, act, 2, 3)) == 0


def test_rows_whose_mask_leaves_nothing():
    m = make(5, [6, 200], 6, 32)
    m["masks"][2] = 0                     # sequence 0 has no context: token 2 sees nothing
    m["masks"][6 + 1] = 0                 # sequence 1: token 1 sees its context alone
    m["masks"][3] = 1 << 5 | 2 ** 63      # bits at and beyond the drafts are ignored
    assert check(m) == 0


def test_more_drafts_than_positions():
    m = make(6, [3, 0, 140], 8, 16, tree=False)
    assert check(m) == 0
    m = make(7, [3, 1], 8, 16, tree=True)
    assert check(m) == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_drafted_row_reaches_only_those_that_see_it(value, int8):
    m = make(8, [300], 6, 16, int8=int8)
    m["masks"] = [1, 3, 5, 9, 19, 37]  # token 2 is seen by 2 and 5
    row = m["table"][0, 296 // 128] * 128 + 296 % 128
    if int8:
        m["scales"][row, 1] = value
    else:
        m["kv_nope"][row, 200] = value
    m["kv_rope"][row, 3] = value
    out, lse, _ = run(m)
    clean = make(8, [300], 6, 16, int8=int8)
    clean["masks"] = m["masks"]
    ref = run(clean)
    for s in (0, 1, 3, 4):
        np.testing.assert_array_equal(out[s], ref[0][s])
        np.testing.assert_array_equal(lse[s], ref[1][s])
    if np.isnan(value):
        assert np.isnan(out[[2, 5]]).all() and np.isnan(lse[[2, 5]]).all()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bad", [-1, -5, 10 ** 6, 2 ** 31 - 1])
def test_bad_pages_are_masked_and_flagged(bad, int8):
    import mla_sparse_top_gb300 as mla
    m = make(9, [700, 300], 4, 32, int8=int8, poison=False)
    m["table"][0, 2] = bad
    assert check(m) == mla.MLA_DEVICE_BAD_BLOCK
    assert mla.tree_device_status() == 0
    m = make(10, [700, 300], 4, 32, int8=int8)
    m["table"][1, 2] = bad  # the page of the drafts
    assert check(m) == mla.MLA_DEVICE_BAD_BLOCK


def test_positions_beyond_the_table_are_masked_and_flagged():
    import mla_sparse_top_gb300 as mla
    m = make(11, [700], 4, 32)
    m["table"] = np.ascontiguousarray(m["table"][:, :4])
    assert check(m) == mla.MLA_DEVICE_BAD_BLOCK


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.4])
def test_scales(scale):
    assert check(make(12, [600, 40], 3, 48, scale=scale)) == 0


def test_out_aligned_to_16_bytes_only_and_nothing_behind_it():
    m = make(20, [700, 3000], 3, 50)
    d = upload(m)
    n = d["q_nope"].numel()
    room = torch.full((n + 24,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[8:8 + n].view(d["q_nope"].shape)
    assert out.data_ptr() % 32 == 16
    lse = torch.empty(out.shape[:2], device="cuda")
    launch(m, d, out, lse)
    check(m, (out.double().cpu().numpy(), lse.double().cpu().numpy(), 0))
    assert (room[:8] == 7).all() and (room[8 + n:] == 7).all()


def test_much_padding_few_sequences():
    m = make(21, [200, 0], 90, 16, lens=[1, 0])
    assert check(m) == 0
    m = make(22, [150] * 200, 4, 64, lens=[b % 5 for b in range(200)])
    assert check(m) == 0


def test_growing_scores_rescale_the_output():
    """Keys that grow along the context: the running maximum rises from tile to tile."""
    m = make(13, [2500], 2, 64, poison=False)
    pos = np.arange(2500)
    rows = m["table"][0, pos // 128] * 128 + pos % 128
    m["kv_nope"][rows] = (m["kv_nope"][rows].float() * torch.linspace(0.1, 3, 2500)[:, None]).bfloat16()
    assert check(m) == 0


def test_other_stream_graph_and_two_graphs_with_workspaces_of_their_own():
    import mla_sparse_top_gb300 as mla
    m, m2 = make(14, [3000], 2, 128), make(15, [2000, 100], 3, 64, int8=True)
    want, want2 = run(m)[0], run(m2)[0]
    d, d2 = upload(m), upload(m2)
    out, out2 = torch.zeros_like(d["q_nope"]), torch.zeros_like(d2["q_nope"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = launch(m, d, out, None, stream=s)
        ws2 = launch(m2, d2, out2, None, stream=s)
    s.synchronize()
    np.testing.assert_array_equal(out.double().cpu().numpy(), want)
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        launch(m, d, out, None, ws)
    with torch.cuda.graph(g2):
        launch(m2, d2, out2, None, ws2)
    out.zero_(), out2.zero_()
    torch.cuda.synchronize()
    t = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            g.replay()
        with torch.cuda.stream(t):
            g2.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out.double().cpu().numpy(), want)
    np.testing.assert_array_equal(out2.double().cpu().numpy(), want2)
    d["act_seqs"].fill_(777)  # another length through the same graph
    g.replay()
    torch.cuda.synchronize()
    m["act"] = np.array([777], np.int32)
    e = step.tree_attention(m["q_nope"].double().numpy(), m["q_rope"].double().numpy(), latent_of(m),
                            m["kv_rope"].double().numpy(), m["table"], m["act"], None, m["masks"], 2, m["scale"])
    assert (np.abs(out.double().cpu().numpy() - e[0]) <= 1.1 * HALF * (e[2] + np.abs(e[0]))).all()
    assert mla.tree_device_status(clear=True) == 0


def test_binding_refuses_what_it_cannot_pass_on():
    m = make(16, [100], 1, 16)
    d = upload(m)
    out, lse = torch.empty_like(d["q_nope"]), torch.empty(d["q_nope"].shape[:2], device="cuda")
    for k, v in (("q_nope", d["q_nope"].half()), ("q_nope", d["q_nope"][:, :, ::2]), ("q_rope", d["q_rope"].cpu()),
                 ("kv_rope", d["kv_rope"][:-128]), ("act_seqs", d["act_seqs"].long()), ("tree_mask", d["act_seqs"]),
                 ("block_table", d["block_table"].t())):
        if k == "block_table" and d[k].shape[0] == d[k].shape[1]:
            continue
        with pytest.raises(ValueError):
            launch(m, {**d, k: v}, out, lse)
