"""Inputs, oracle runs and error bounds of the operators on ordinary heads.

Bound of one attention output, with u = 2^-24 (half a step of fp32), p the softmax and n the keys:
a score's products are exact; its sum of D terms, each addition off by at most a step of fp32 (the
tensor cores may truncate), and the products with the scale, the maximum's subtraction and 2^x (two
steps) leave it off by dz = 2 u D terms + 8 u (|z| + 1), terms the largest sum of |q_d k_d| scale.
That moves every weight by a factor of at most 1 + 2 dz (the maximum's own error goes into all of
them alike).  A weight is rounded to the heads' type once (eps / 2 of it; fp16 below its normal range by 2^-25 at
most, where the largest weight is at least 1), the sums over n keys add n steps, and the
merge of parts 16 u.  All of that times sum_p p |v|, and half a step of the output's type.
"""
import numpy as np
import torch

from oracle import heads

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def cache(blocks, Hkv, D, layout, dtype, fill=None, gen=None):
    """(blocks, 128, Hkv, D) on the GPU, its memory by token, by head, or keys and values sharing pages."""
    if layout == "head":
        x = torch.empty((blocks, Hkv, 128, D), dtype=dtype, device="cuda").transpose(1, 2)
    elif layout == "shared":  # every second run of a page of twice the heads
        x = torch.empty((blocks, 128, 2, Hkv, D), dtype=dtype, device="cuda")[:, :, 0]
    else:
        x = torch.empty((blocks, 128, Hkv, D), dtype=dtype, device="cuda")
    if fill is not None:
        x.fill_(fill)
    else:
        x.copy_(torch.randn(x.shape, generator=gen).to(dtype))
    return x


def normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen).to(dtype).cuda()


def padded(gen, T, H, D, dtype, pad=0):
    """(T, H, D), a view with gaps between tokens and heads."""
    return normal(gen, (T, H + (1 if pad else 0), D + pad), dtype)[:, :H, :D]


def page_table(gen, act, W=None, spare=2):
    """A pool in which the sequences' pages lie anywhere; entries behind them are garbage ids."""
    need = [-(-a // 128) for a in act]
    used = sum(need) + spare
    perm = torch.randperm(used, generator=gen)
    W = max([1] + need) if W is None else W
    table = torch.full((len(act), W), 123456789, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :min(n, W)] = perm[at:at + n][:W].to(torch.int32)
        at += n
    return table, used


def np64(x):
    return x.detach().double().cpu().numpy()


def check_rows(got, got_lse, ref, dtype, keys, what):
    out, lse, mass, terms, top = ref
    got, got_lse = np64(got), np64(got_lse)
    info = torch.finfo(dtype)
    D = check_rows.D
    dz = 2 * U * D * terms + 8 * U * (top + 1)
    rel = info.eps / 2 + 2 * dz[..., None] + 2 * U * (keys + 16)
    bound = mass * rel * (1 + 1e-3) + np.maximum(np.abs(out), info.smallest_normal) * info.eps / 2
    if dtype == torch.float16:
        bound = bound + keys * check_rows.vmax * 2.0 ** -25
    dead = np.isneginf(lse)
    assert (np.isneginf(got_lse) == dead).all(), what
    assert (got[dead] == 0).all(), what
    err = np.abs(got - out)
    assert (err <= bound).all(), f"{what}: worst {np.nanmax(err / bound)} at {np.unravel_index(np.nanargmax(err / bound), err.shape)}, finite {np.isfinite(got).all()}"
    lb = dz + 2 * U * (keys + 16) + 4 * U * np.abs(np.where(dead, 0, lse))
    le = np.abs(np.where(dead, 0, got_lse) - np.where(dead, 0, lse))
    assert (le <= lb).all(), f"{what}: lse worst {np.nanmax(le / lb)}"


def check_sequence(got, got_lse, q, k, v, scale, causal, what, seen=None):
    """One sequence's rows against the oracle, in blocks of queries."""
    check_rows.D = q.shape[2]
    n, L = q.shape[0], k.shape[0]
    k64, v64 = np64(k), np64(v)
    check_rows.vmax = np.abs(v64).max(initial=0)
    size = max(1, 40_000_000 // max(1, L * q.shape[1]))
    for s in range(0, n, size):
        e = min(n, s + size)
        end = max(0, L - n + e) if causal else L  # keys that this block may see
        ref = heads.attention(np64(q[s:e]), k64[:end], v64[:end], scale, causal, None if seen is None else seen[:end])
        check_rows(got[s:e], got_lse[s:e], ref, got.dtype, L, f"{what} rows {s}")


def gather(pool, table, b, length):
    """The first `length` keys of sequence b."""
    pages = table[b, :-(-length // 128)].long()
    return pool.cpu()[pages].flatten(0, 1)[:length]


def check_gpu(got, got_lse, q, k, v, scale, causal, what):
    """check_sequence on the GPU in fp64, head by head, for sequences that numpy takes too long over."""
    n, H, D = q.shape
    L, Hkv = k.shape[:2]
    if n == 0 or L == 0:
        assert (got == 0).all() and torch.isneginf(got_lse).all(), what
        return
    info = torch.finfo(got.dtype)
    vmax = v.abs().max().double().item()
    for h in range(H):
        a, b, c = q[:, h].double(), k[:, h * Hkv // H].double(), v[:, h * Hkv // H].double()
        z = a @ b.T * scale
        hidden = torch.arange(L, device=q.device)[None] > (L - n + torch.arange(n, device=q.device))[:, None] if causal else \
            torch.zeros((n, L), dtype=torch.bool, device=q.device)
        z.masked_fill_(hidden, -float("inf"))
        lse = torch.logsumexp(z, -1)
        p = (z - lse[:, None]).exp()
        out, mass = p @ c, p @ c.abs()
        top = z.abs().masked_fill(hidden, 0).amax(-1)
        terms = (a.abs() @ b.abs().T * abs(scale)).masked_fill(hidden, 0).amax(-1)
        dz = 2 * U * D * terms + 8 * U * (top + 1)
        bound = mass * (info.eps / 2 + 2 * dz[:, None] + 2 * U * (L + 16)) * (1 + 1e-3)
        bound = bound + out.abs().clamp(min=info.smallest_normal) * info.eps / 2
        if got.dtype == torch.float16:
            bound = bound + L * vmax * 2.0 ** -25
        err = (got[:, h].double() - out).abs()
        assert bool((err <= bound).all()), f"{what} head {h}: worst {(err / bound).max().item()}, finite {bool(torch.isfinite(got[:, h]).all())}"
        le = (got_lse[:, h].double() - lse).abs()
        assert bool((le <= dz + 2 * U * (L + 16) + 4 * U * lse.abs()).all()), f"{what} head {h}: lse {le.max().item()}"
