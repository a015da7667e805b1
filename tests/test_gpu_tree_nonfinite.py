"""Infinities in cache rows, against the formula: a weight of 0 times an
infinite value is NaN, in that value's output column alone, for the tokens that
see the row, whether it is a drafted one or not and whether the row block was
cut between clusters or not.  Expectations are built from the scores one key at
a time; bounds of finite outputs are those of test_gpu_tree.py."""
import numpy as np
import pytest
import torch

from oracle import step
from test_gpu_tree import HALF, U, latent_of, make, run

pytestmark = pytest.mark.gpu


def row_of(m, b, pos):
    return m["table"][b, pos // 128] * 128 + pos % 128


def one_sided(m, cols):
    """Queries of these columns above 0 for even heads and below for odd ones: an infinite score gets one sign."""
    q = m["q_nope"][:, :, cols].float().abs() + 0.125
    q[:, 1::2] *= -1
    m["q_nope"][:, :, cols] = q.bfloat16()


def spoil(m, b, pos, value, col):
    """An infinity in column `col` of one row; in the whole scale group of an INT8 row."""
    row = row_of(m, b, pos)
    if m["scales"] is None:
        m["kv_nope"][row, col] = value
        return
    group = slice(col // 128 * 128, col // 128 * 128 + 128)
    m["kv_nope"][row, group] = m["kv_nope"][row, group].float().abs().clamp(1, 127).to(torch.int8)
    m["scales"][row, col // 128] = value


def expected(m, lat):
    qn, qr, rope = (m[k].double().numpy() for k in ("q_nope", "q_rope", "kv_rope"))
    T, H, D = qn.shape
    out, mag, lse = np.zeros((T, H, D)), np.zeros((T, H, D)), np.full((T, H), -np.inf)
    for t in range(T):
        b, s = divmod(t, m["S1"])
        seen = step.tree_visible(m["act"][b], m["S1"], s, None if m["masks"] is None else m["masks"][t])
        rows = np.array([row_of(m, b, p) for p in seen], dtype=np.int64)
        v = lat[rows]
        odd = ~np.isfinite(v).all(1)
        z = np.empty((H, len(rows)))
        z[:, ~odd] = m["scale"] * (qn[t] @ v[~odd].T + qr[t] @ rope[rows[~odd]].T)
        with np.errstate(invalid="ignore"):
            for i in np.flatnonzero(odd):
                z[:, i] = m["scale"] * ((qn[t] * v[i]).sum(-1) + qr[t] @ rope[rows[i]])
        for h in range(H):
            if np.isnan(z[h]).any() or np.isposinf(z[h]).any():
                out[t, h], lse[t, h] = np.nan, np.nan
                continue
            keep = np.isfinite(z[h])
            if not keep.any():
                continue
            top = z[h, keep].max()
            e = np.exp(z[h, keep] - top)
            out[t, h], mag[t, h] = e @ v[keep] / e.sum(), e @ np.abs(v[keep]) / e.sum()
            lse[t, h] = top + np.log(e.sum())
            out[t, h, ~np.isfinite(v[~keep]).all(0)] = np.nan
    return out, lse, mag


def check(m):
    out, lse, status = run(m)
    assert status == 0
    lat = latent_of(m)
    o, e, mag = expected(m, lat)
    keys = np.concatenate([np.where(np.isfinite(lat), lat, 0), np.nan_to_num(m["kv_rope"].double().numpy())], 1)
    q = np.concatenate([m["q_nope"].double().numpy(), m["q_rope"].double().numpy()], -1)
    top = float(np.linalg.norm(keys, axis=1).max() * np.linalg.norm(q, axis=-1).max())
    d = abs(m["scale"]) * top * 578 * U + (int(m["act"].max()) + 16) * U
    assert (np.isnan(out) == np.isnan(o)).all(), f"{(np.isnan(out) != np.isnan(o)).sum()} of {o.size} outputs"
    ok = ~np.isnan(o)
    bound = (HALF + 2 * d) * mag * (1 + 2 * d) + HALF * np.abs(o) * 1.01 + 1e-30
    assert (np.abs(out - o)[ok] <= bound[ok]).all()
    assert (np.isnan(lse) == np.isnan(e)).all() and (np.isneginf(lse) == np.isneginf(e)).all()
    fin = np.isfinite(e)
    assert (np.abs(lse[fin] - e[fin]) <= d + 4 * U * (1 + np.abs(e[fin]))).all()
    return o, e


# one row block, a row block cut among a few clusters and among many, several row blocks (INT8: rows expanded first)
SHAPES = [dict(act=[300], S1=6, n_q=16), dict(act=[9000], S1=2, n_q=64), dict(act=[700, 20000], S1=3, n_q=5, W=700),
          dict(act=[300, 1000], S1=4, n_q=128)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_drafted_infinity_gives_what_the_formula_gives(shape, tree, value, int8):
    m = make(40, int8=int8, tree=tree, **shape)
    one_sided(m, slice(128, 256))
    b, S1 = len(m["act"]) - 1, m["S1"]
    j = S1 // 2
    if tree:  # the last token sees it, the one before does not
        m["masks"][b * S1 + S1 - 1] |= 1 << j
        if S1 - 2 != j:
            m["masks"][b * S1 + S1 - 2] &= ~(1 << j)
    spoil(m, b, int(m["act"][b]) - S1 + j, value, 200)
    o, e = check(m)
    last = o[b * S1 + S1 - 1]
    # half of the heads score -inf there: they lose that column, or group of columns, alone
    some = np.isnan(last).any(-1) & ~np.isnan(last).all(-1)
    assert some.sum() == m["q_nope"].shape[1] // 2 or m["q_nope"].shape[1] % 2
    assert np.isnan(last[:, 200]).all() and np.isfinite(o[b * S1]).all()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("act,S1", [(9000, 1), (9000, 2), (20000, 1)])
def test_context_infinities_survive_the_merge(act, S1, int8):
    """Every key of one tile scores -inf for half of the heads: a part in which their weights are all 0."""
    m = make(41, [act], S1, 16, int8=int8, tree=False, W=700)
    one_sided(m, slice(0, 128))
    for pos in range(1024, 1280):
        spoil(m, 0, pos, float("inf"), 7)
    o, _ = check(m)
    assert np.isnan(o[:, 1::2, 7]).all() and np.isfinite(o[:, 1::2, 200]).all()


@pytest.mark.parametrize("int8", [False, True])
def test_a_part_of_drafts_alone_that_all_score_minus_infinity(int8):
    m = make(42, [8192 + 4], 4, 16, int8=int8, tree=False, W=700)
    one_sided(m, slice(128, 256))
    for j in range(4):
        spoil(m, 0, 8192 + j, float("inf"), 130)
    check(m)


def test_tokens_whose_every_score_is_minus_infinity():
    """Counted like tokens that see nothing: no output, lse -inf."""
    m = make(43, [5], 5, 16, tree=False)
    one_sided(m, slice(128, 256))
    for j in range(5):
        spoil(m, 0, j, float("inf"), 150)
    o, e = check(m)
    assert (o[:, 1::2] == 0).all() and np.isneginf(e[:, 1::2]).all() and np.isnan(o[:, ::2]).all()


@pytest.mark.parametrize("int8", [False, True])
def test_a_rope_infinity_with_a_finite_latent_changes_no_column(int8):
    m = make(44, [300], 4, 16, int8=int8, tree=False)
    q = m["q_rope"][:, :, 9].float().abs() + 0.125
    q[:, 1::2] *= -1
    m["q_rope"][:, :, 9] = q.bfloat16()
    m["kv_rope"][row_of(m, 0, 297), 9] = float("inf")
    out, lse, _ = run(m)
    assert np.isfinite(out[:, 1::2]).all() and np.isfinite(lse[:, 1::2]).all()
    assert np.isnan(out[1:, ::2]).all() and np.isfinite(out[0]).all()


@pytest.mark.parametrize("int8", [False, True])
def test_rows_of_a_cut_block_whose_mask_leaves_nothing(int8):
    """No context, drafts over two tiles, a team for each: both parts of those rows hold nothing."""
    m = make(45, [300], 300, 2, int8=int8, W=700)
    for s in (0, 5, 70, 299):
        m["masks"][s] = 0
    m["masks"][298] = 1 << 290  # the first tile holds nothing
    o, e = check(m)
    assert (o[[0, 5, 70, 299]] == 0).all() and np.isneginf(e[[0, 5, 70, 299]]).all() and np.isfinite(e[298]).all()
