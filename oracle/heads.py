"""fp64 oracle of the operators on ordinary heads (include/mla_heads.h), written from their definitions."""
import numpy as np

from oracle import step


def norm(x, kind, weight=None, bias=None, eps=1e-6):
    """Norm of each head over its last axis; kind None, "rms" or "layer"."""
    x = np.asarray(x, np.float64)
    if kind is None:
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y


def norm_rope(x, positions, kind, weight, bias, eps, freqs, *, rot_off, half, mscale=1.0):
    """x (T, H, D): norm, then the rotation of the pairs that freqs has (none for no frequencies)."""
    y = norm(x, kind, weight, bias, eps)
    if len(freqs) == 0:
        return y
    return step.rope_apply(y, positions, freqs, rot_off=rot_off, half=half, inverse=False, mscale=mscale)


def append(cache, rows, x):
    """cache (blocks, 128, H, D) with the tokens x (T, H, D) at rows; rows outside it are left out."""
    flat = np.array(cache).reshape(-1, *cache.shape[2:])
    for t, r in enumerate(rows):
        if 0 <= r < len(flat):
            flat[r] = x[t]
    return flat.reshape(cache.shape)


def attention(q, k, v, scale, causal, seen=None):
    """One sequence: q (n, H, D), k (len, Hkv, D), v (len, Hkv, Dv), the queries its newest tokens.

    Returns out (n, H, Dv), lse (n, H), and with them sum_p softmax_p |v_p|, the largest sum_d |q_d k_d|
    scale of a score that a token sees and its largest |score|, which error bounds are made of.  `seen`
    (len,): keys that exist at all."""
    n, H = q.shape[:2]
    L, Hkv = k.shape[:2]
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    g = H // Hkv
    kk, vv = np.repeat(k, g, 1), np.repeat(v, g, 1)
    vis = np.ones((n, L), bool)
    if causal:
        vis = np.arange(L)[None] <= (L - n + np.arange(n))[:, None]
    if seen is not None:
        vis = vis & seen[None]
    with np.errstate(all="ignore"):
        z = np.einsum("nhd,lhd->hnl", q, kk) * scale
        z = np.where(vis[None], z, -np.inf)
        m = z.max(-1, initial=-np.inf)
        e = np.where(vis[None], np.exp(z - np.where(np.isinf(m), 0, m)[..., None]), 0)
        s = e.sum(-1)
        p = e / np.where(s == 0, 1, s)[..., None]
        out = np.einsum("hnl,lhd->nhd", p, vv)
        mass = np.einsum("hnl,lhd->nhd", p, np.abs(vv))
        terms = np.einsum("nhd,lhd->hnl", np.abs(q), np.abs(kk)) * abs(scale)
        lse = m + np.log(s)
        terms = np.where(vis[None], terms, 0).max(-1, initial=0)
        top = np.where(vis[None], np.abs(z), 0).max(-1, initial=0)
    return out, lse.T, mass, terms.T, top.T
