"""Oracles of the calls around a drafted decode step, in plain Python and
numpy fp64: the page plan (block tables, slot maps, positions, tree masks) and
rotary positions.  Test infrastructure only; written from the formulas, one
request, token and pair at a time."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 128
NO_PAGE, BAD_BLOCK = 0x4, 0x1


def page_plan(ctx_lens, new_lens, free_blocks, block_table, *, S1, T, num_blocks, parents=None):
    """The outputs of mla_page_plan as a dict (tree_mask as Python integers)."""
    B, W = block_table.shape
    table = block_table.copy()
    act, cu, taken, status = [], [0], 0, 0
    idx, pos, seq, mask = [-1] * T, [0] * T, [-1] * T, [0] * T
    nf = len(free_blocks)
    for b in range(B):
        ctx = max(0, int(ctx_lens[b]))
        new = S1 if new_lens is None else max(0, int(new_lens[b]))
        if S1:
            new = min(new, S1)
        have, total = min(W, -(-ctx // BLOCK)), min(W, -(-(ctx + new) // BLOCK))
        for w in range(have, total):
            if taken < nf:
                table[b, w] = free_blocks[taken]
            else:
                table[b, w] = -1
                status |= NO_PAGE
            taken += 1
        up = []
        for i in range(new):
            t = b * S1 + i if S1 else cu[-1] + i
            if parents is not None:
                par = int(parents[b][i])
                up.append((up[par] if 0 <= par < i else 0) | 1 << i)
            else:
                up.append((2 << i) - 1)
            if t >= T:
                status |= NO_PAGE
                continue
            slot = ctx + i
            if slot // BLOCK >= W:
                status |= NO_PAGE
            else:
                blk = int(table[b, slot // BLOCK])
                fresh = slot // BLOCK >= have
                if 0 <= blk < num_blocks:
                    idx[t] = blk * BLOCK + slot % BLOCK
                elif not (fresh and blk == -1 and status & NO_PAGE):
                    status |= BAD_BLOCK
            pos[t], seq[t], mask[t] = ctx + bin(up[i]).count("1") - 1, b, up[i]
        act.append(ctx + new)
        cu.append(cu[-1] + new)
    return dict(block_table=table, act_seqs=np.array(act), cu_seqs=np.array(cu), num_taken=min(taken, nf),
                cache_index=np.array(idx), positions=np.array(pos), seq_ids=np.array(seq), tree_mask=mask,
                status=status)


def rope_freqs(rot_dim, theta=10000.0, scaling="none", factor=1.0, orig_positions=4096, beta_fast=32.0,
               beta_slow=1.0):
    """Angle per position of each pair."""
    out = []
    base = theta * factor ** (rot_dim / max(rot_dim - 2, 1)) if scaling == "ntk" else theta
    for i in range(rot_dim // 2):
        f = base ** (-2 * i / rot_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            def dim_of(beta):
                return rot_dim * math.log(orig_positions / (2 * math.pi * beta)) / (2 * math.log(base))
            low, high = max(math.floor(dim_of(beta_fast)), 0), min(math.ceil(dim_of(beta_slow)), rot_dim - 1)
            r = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            f = f * (1 - r) + f / factor * r
        out.append(f)
    return np.array(out)


def rope_apply(x, positions, freqs, *, rot_off, half, inverse=False, mscale=1.0):
    """x (T, H, D) fp64 with the pairs of [rot_off, rot_off + 2 len(freqs)) turned by positions * freqs."""
    y = np.array(x, dtype=np.float64)
    n = len(freqs)
    for i, f in enumerate(freqs):
        a = np.asarray(positions, dtype=np.float64) * f
        c, s = mscale * np.cos(a)[:, None], mscale * np.sin(a)[:, None] * (-1 if inverse else 1)
        p, q = (rot_off + i, rot_off + i + n) if half else (rot_off + 2 * i, rot_off + 2 * i + 1)
        u, v = x[:, :, p], x[:, :, q]
        y[:, :, p], y[:, :, q] = u * c - v * s, u * s + v * c
    return y


def tree_visible(act, n, s, mask_bits):
    """Positions of one sequence that drafted token s (of n) sees; mask_bits: its tree_mask row as an integer, or None."""
    act = max(0, int(act))
    if s >= n:
        return []
    ctx = act - n
    bits = (2 << s) - 1 if mask_bits is None else mask_bits
    return [p for p in range(act) if p < ctx or bits >> (p - ctx) & 1]


def tree_attention(q_nope, q_rope, latent, rope, block_table, act_seqs, tree_lens, masks, S1, scale):
    """fp64: q_nope (T, H, 512), q_rope (T, H, 64), latent (rows, 512) and rope
    (rows, 64) as fp64 values, masks: T integers or None.  Returns out, lse and
    sum_p softmax_p |v_p| (what a rounding of the weights acts on)."""
    T, H, D = q_nope.shape
    out, mag = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    num_blocks = latent.shape[0] // BLOCK
    for t in range(T):
        b, s = divmod(t, S1)
        n = S1 if tree_lens is None else min(S1, max(0, int(tree_lens[b])))
        rows = []
        for p in tree_visible(act_seqs[b], n, s, None if masks is None else masks[t]):
            blk = int(block_table[b, p // BLOCK]) if p // BLOCK < block_table.shape[1] else -1
            if 0 <= blk < num_blocks:
                rows.append(blk * BLOCK + p % BLOCK)
        if not rows:
            continue
        v = latent[rows]
        z = scale * (q_nope[t] @ v.T + q_rope[t] @ rope[rows].T)
        m = z.max(-1, keepdims=True)
        e = np.exp(z - m)
        l = e.sum(-1, keepdims=True)
        out[t], mag[t] = e / l @ v, e / l @ np.abs(v)
        lse[t] = (m + np.log(l))[:, 0]
    return out, lse, mag
