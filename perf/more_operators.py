"""Grouped-head attention beside the latent one, as cases to measure: norms and rotation of heads, the write of keys
and values into a paged cache, attention over whole prompts and attention of new tokens over the pages.

`run` computes the plain form in elementary torch operations, or, where `own` is true, makes the calls that a user
makes of the library. Heads are (tokens, heads, values) tensors; a paged cache is (blocks, 128, heads, values), its
memory ordered by token or by head.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
_TYPES = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the indexer's queries (rotated alone) and its new keys (LayerNorm, then rotated) of a decode step, the keys
        # written to their cache rows: latency
        dict(name="norm_index_keys", op="norm", T=128, H=64, D=128, off=0, rot=64, half=True, q_norm="none", K=1,
             k_norm="layer", rows=True, dtype="bf16", scaling="yarn", factor=40.0, maxpos=163840, pad=0),
        # queries and keys of a prompt chunk, RMS norms and the whole head rotated: the ordinary case
        dict(name="norm_prompt", op="norm", T=8192, H=32, D=128, off=0, rot=128, half=True, q_norm="rms", K=8,
             k_norm="rms", rows=False, dtype="bf16", scaling="none", factor=1.0, maxpos=8192, pad=0),
        # odd sizes in fp32, padded strides, part of the head turned, far positions
        dict(name="norm_odd", op="norm", T=4099, H=17, D=107, off=7, rot=36, half=False, q_norm="layer", K=0,
             k_norm="none", rows=False, dtype="fp32", scaling="linear", factor=8.0, maxpos=1 << 20, pad=5),
        # 64 new tokens of a decode step into a cache ordered by token: latency
        dict(name="append_decode", op="append", T=64, H=32, Hkv=8, D=128, Dv=128, rot=128, half=True, q_norm="rms",
             k_norm="rms", layout="token", dtype="bf16", skip=3),
        # a prompt chunk into a cache ordered by head, without norms
        dict(name="append_prompt", op="append", T=16384, H=28, Hkv=4, D=128, Dv=128, rot=64, half=False,
             q_norm="none", k_norm="none", layout="head", dtype="fp16", skip=0),
        # one short prompt: latency
        dict(name="prompt_small", op="prompt", B=1, lo=300, hi=300, ctx_lo=0, ctx_hi=0, H=16, Hkv=4, D=64, Dv=64,
             dtype="bf16", paged=False, causal=True, layout="token", spare=0),
        # prompts of 1 to 2500 tokens packed behind one another, rows left over behind the last
        dict(name="prompt_packed", op="prompt", B=9, lo=1, hi=2500, ctx_lo=0, ctx_hi=0, H=32, Hkv=8, D=128, Dv=128,
             dtype="bf16", paged=False, causal=True, layout="token", spare=37),
        # a long prompt of latent attention before absorption, 192 values to a key and 128 to a value: the largest
        dict(name="prompt_latent", op="prompt", B=1, lo=8192, hi=8192, ctx_lo=0, ctx_hi=0, H=128, Hkv=128, D=192,
             Dv=128, dtype="bf16", paged=False, causal=True, layout="token", spare=0),
        # chunks of long prompts over what their pages hold already, seven queries to a key head
        dict(name="prompt_chunk", op="prompt", B=3, lo=257, hi=300, ctx_lo=5000, ctx_hi=60000, H=28, Hkv=4, D=128,
             Dv=128, dtype="fp16", paged=True, causal=True, layout="head", spare=0),
        # one request of a small model, one token: latency
        dict(name="paged_one_request", op="paged", B=1, S1=1, lo=1000, hi=1000, H=16, Hkv=2, D=64, Dv=64,
             dtype="bf16", layout="token", ragged=False),
        # a decode batch, every length another
        dict(name="paged_batch", op="paged", B=64, S1=1, lo=100, hi=8192, H=32, Hkv=8, D=128, Dv=128, dtype="bf16",
             layout="token", ragged=False),
        # chains of up to five drafted tokens, padding rows among them, a head size that is no power of two
        dict(name="paged_chains", op="paged", B=24, S1=5, lo=500, hi=20000, H=40, Hkv=8, D=96, Dv=96, dtype="fp16",
             layout="head", ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "prompt", "prompt", "paged", "paged"])
    if op == "norm":
        rot = rng.choice([0, 64, 64, 128, 2 * rng.randint(1, 100)])
        off = rng.choice([0, 0, 64, rng.randint(0, 60)])
        D = max(1, off + rot + rng.choice([0, 0, 64, rng.randint(0, 70)]))
        T, H, K = _log(rng, 1, 20000), rng.choice([1, 3, 16, 32, 64]), rng.choice([0, 1, 4, 8])
        while T * (H + K) * D > 30_000_000:
            T = T // 2
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op="norm", T=T, H=H, D=D, off=off, rot=rot, half=rng.random() < 0.5,
                    q_norm=rng.choice(["none", "rms", "rms", "layer"]), K=K, k_norm=rng.choice(["rms", "rms", "layer"]),
                    rows=K > 0 and rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 40.0]),
                    maxpos=_log(rng, 100, 1 << 20), pad=rng.choice([0, 0, 8, 3]))
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    D = rng.choice([64, 96, 128, 128, 8 * rng.randint(1, 16), 192])
    Dv = 128 if D == 192 else rng.choice([D, D, 8 * rng.randint(1, 16)])
    dtype, layout = rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["token", "head"])
    heads = dict(H=G * Hkv, Hkv=Hkv, D=D, Dv=Dv, dtype=dtype, layout=layout)
    if op == "append":
        T = _log(rng, 1, 16384)
        while T * (G * Hkv + Hkv) * D > 60_000_000:
            T = T // 2
        rot = rng.choice([0, min(D, 64), D, 2 * rng.randint(1, D // 2)])
        return dict(op="append", T=T, rot=rot, half=rng.random() < 0.5, q_norm=rng.choice(["none", "rms", "layer"]),
                    k_norm=rng.choice(["none", "rms", "layer"]), skip=rng.choice([0, T // 7]), **heads)
    if op == "prompt":
        B, hi = _log(rng, 1, 40), _log(rng, 1, 8192)
        paged = rng.random() < 0.4
        ctx = rng.choice([0, _log(rng, 1, 60000)]) if paged else 0
        while B * G * Hkv * hi * (hi + ctx) > (1 << 32) or B * (hi + ctx) * Hkv * (D + Dv) > (1 << 28) \
                or B * hi * G * Hkv * D > (1 << 26):
            B, hi, ctx = max(1, B * 2 // 3), max(1, hi * 2 // 3), ctx * 2 // 3
        return dict(op="prompt", B=B, lo=rng.choice([1, 1 + hi // 3, hi]), hi=hi, ctx_lo=rng.choice([0, ctx]), ctx_hi=ctx,
                    paged=paged, causal=rng.random() < 0.85, spare=rng.choice([0, 19]), **heads)
    S1, B, hi = rng.choice([1, 1, 1, 2, 5, 8]), _log(rng, 1, 128), _log(rng, 1, 60000)
    while B * hi * Hkv * (D + Dv) > (1 << 28):
        B, hi = max(1, B * 2 // 3), max(1, hi * 2 // 3)
    return dict(op="paged", B=B, S1=S1, lo=rng.choice([1, 1 + hi // 40, hi]), hi=hi, ragged=rng.random() < 0.4, **heads)


def _spread(n, lo, hi, turn=0.6180339887498949):
    """n lengths between lo and hi, even in their logarithm, in no order (the same ones for every seed)."""
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [max(lo, min(hi, int(round(math.exp(a + (b - a) * ((i + 1) * turn % 1.0)) - 1)))) for i in range(n)]


def _new_tokens(case):
    """New tokens of each sequence."""
    if case["op"] == "prompt":
        return _spread(case["B"], case["lo"], case["hi"])
    if not case["ragged"]:
        return [case["S1"]] * case["B"]
    return [int(case["S1"] * (((i + 1) * 0.7548776662466927) % 1.0) + 0.5) for i in range(case["B"])]


def _lengths(case):
    """(new tokens, keys) of each sequence."""
    new = _new_tokens(case)
    if case["op"] == "prompt":
        ctx = _spread(case["B"], case["ctx_lo"], case["ctx_hi"], 0.7548776662466927)
    else:
        ctx = _spread(case["B"], case["lo"], case["hi"])
    return new, [n + c for n, c in zip(new, ctx)]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _cumulative(lens):
    return _ints([0] + lens, torch.int64).cumsum(0).to(torch.int32)


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _scheme(case):
    """The frequency scheme that a model's configuration gives."""
    scaling, factor = case.get("scaling", "none"), case.get("factor", 1.0)
    return dict(theta=10000.0, scaling=scaling, factor=factor, orig_positions=4096, beta_fast=32.0, beta_slow=1.0,
                mscale=0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def _norm(g, kind, D, dtype):
    """(kind, weight, bias): weights around one, in the heads' type, LayerNorm's in fp32 as they are stored."""
    if kind == "none":
        return None
    weight = torch.rand((D,), generator=g, device="cuda") + 0.5
    if kind == "rms":
        return kind, weight.to(dtype), None
    return kind, weight, torch.randn((D,), generator=g, device="cuda") / 4


def _prepare_norm(case, seed):
    g = _gen(seed)
    T, dtype, D = case["T"], _TYPES[case["dtype"]], case["D"]
    st = dict(op="norm", rot=case["rot"], off=case["off"], half=case["half"], scheme=_scheme(case), k=None, rows=None,
              positions=torch.randint(0, case["maxpos"], (T,), generator=g, device="cuda", dtype=torch.int32),
              q=_normal(g, (T, case["H"], D + case["pad"]), dtype)[:, :, :D], q_norm=_norm(g, case["q_norm"], D, dtype))
    st["q_out"] = torch.zeros((T, case["H"], D), device="cuda", dtype=dtype)
    if case["K"]:
        st["k"] = _normal(g, (T, case["K"], D + case["pad"]), dtype)[:, :, :D]
        st["k_norm"] = _norm(g, case["k_norm"], D, dtype)
        n = 2 * T if case["rows"] else T
        st["k_out"] = torch.zeros((n, case["K"], D), device="cuda", dtype=dtype)
        if case["rows"]:  # each key's row of its cache
            st["rows"] = torch.randperm(n, generator=g, device="cuda")[:T].contiguous()
    return st


def _cache(blocks, Hkv, D, layout, dtype, g=None):
    """(blocks, 128, heads, values), its memory ordered by token or by head."""
    shape = (blocks, BLOCK, Hkv, D) if layout == "token" else (blocks, Hkv, BLOCK, D)
    x = torch.zeros(shape, device="cuda", dtype=dtype) if g is None else torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    return x if layout == "token" else x.transpose(1, 2)


def _prepare_append(case, seed):
    g = _gen(seed)
    T, H, Hkv, D, Dv, dtype = case["T"], case["H"], case["Hkv"], case["D"], case["Dv"], _TYPES[case["dtype"]]
    blocks = 1 + T * 3 // (2 * BLOCK)
    # queries, keys and values as one product gives them, behind one another
    fused = _normal(g, (T, H * D + Hkv * D + Hkv * Dv), dtype)
    q, k, v = fused.split((H * D, Hkv * D, Hkv * Dv), 1)
    rows = torch.randperm(blocks * BLOCK, generator=g, device="cuda")[:T]
    rows[:case["skip"]] = -1  # padding of the batch
    return dict(op="append", rot=case["rot"], off=0, skip=case["skip"], half=case["half"], scheme=_scheme(case), rows=rows.contiguous(),
                positions=torch.randint(0, 32768, (T,), generator=g, device="cuda", dtype=torch.int32),
                q=q.unflatten(1, (H, D)), k=k.unflatten(1, (Hkv, D)), v=v.unflatten(1, (Hkv, Dv)),
                q_norm=_norm(g, case["q_norm"], D, dtype), k_norm=_norm(g, case["k_norm"], D, dtype),
                q_out=torch.zeros((T, H, D), device="cuda", dtype=dtype),
                k_cache=_cache(blocks, Hkv, D, case["layout"], dtype), v_cache=_cache(blocks, Hkv, Dv, case["layout"], dtype))


def _pages(g, seed, case, act):
    """A pool in which every sequence's pages lie anywhere, and its block table."""
    blocks = [-(-a // BLOCK) for a in act]
    W, used = max(1, max(blocks)), max(1, sum(blocks))
    perm = torch.randperm(used, generator=torch.Generator().manual_seed(int(seed))).to(torch.int32)
    start = torch.tensor([0] + blocks, dtype=torch.int64).cumsum(0)[:len(act), None]
    w = torch.arange(W)[None]
    mine = w < torch.tensor(blocks)[:, None]
    table = torch.where(mine, perm[(start + w).clamp(max=used - 1)], torch.full((len(act), W), -1, dtype=torch.int32))
    dtype = _TYPES[case["dtype"]]
    return dict(block_table=table.cuda(), act_seqs=_ints(act), k=_cache(used, case["Hkv"], case["D"], case["layout"], dtype, g),
                v=_cache(used, case["Hkv"], case["Dv"], case["layout"], dtype, g))


def _prepare_attention(case, seed):
    g = _gen(seed)
    new, act = _lengths(case)
    dtype, H, Hkv, D, Dv = _TYPES[case["dtype"]], case["H"], case["Hkv"], case["D"], case["Dv"]
    paged = case["op"] == "paged"
    T = case["B"] * case["S1"] if paged else sum(new) + case["spare"]
    st = dict(op=case["op"], q=torch.randn((T, H, D), generator=g, device="cuda", dtype=dtype), block_table=None,
              max_q=case["S1"] if paged else max(new), max_k=max(act), scale=D ** -0.5,
              causal=paged or case["causal"])
    if paged:
        st.update(S1=case["S1"], q_lens=_ints(new) if case["ragged"] else None)
    else:
        st.update(cu_q=_cumulative(new))
    if paged or case["paged"]:
        st.update(_pages(g, seed, case, act))
    else:
        st.update(k=torch.randn((T, Hkv, D), generator=g, device="cuda", dtype=dtype),
                  v=torch.randn((T, Hkv, Dv), generator=g, device="cuda", dtype=dtype))
    # rows that the call leaves alone stay as they are here
    st["out"] = torch.zeros((T, H, Dv), device="cuda", dtype=dtype)
    st["lse"] = torch.zeros((T, H), device="cuda", dtype=torch.float32)
    return st


def prepare(case, seed):
    if case["op"] == "norm":
        return _prepare_norm(case, seed)
    if case["op"] == "append":
        return _prepare_append(case, seed)
    return _prepare_attention(case, seed)


# ------------------------------------------------------------------ plain forms
def _inv_freq(scheme, rot, device):
    """Angle per position of each pair, in 64 bits."""
    i = torch.arange(rot // 2, device=device, dtype=torch.float64)
    theta, factor = scheme["theta"], scheme["factor"]
    if scheme["scaling"] == "ntk":
        theta = theta * factor ** (rot / max(rot - 2, 1))
    f = torch.exp(-math.log(theta) * 2 * i / rot)
    if scheme["scaling"] == "linear":
        f = f / factor
    if scheme["scaling"] == "yarn":
        # pairs that turn often over the trained length keep their angle, those that turn rarely are stretched
        low = rot * math.log(scheme["orig_positions"] / (2 * math.pi * scheme["beta_fast"])) / (2 * math.log(theta))
        high = rot * math.log(scheme["orig_positions"] / (2 * math.pi * scheme["beta_slow"])) / (2 * math.log(theta))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
    return f


def _normed(x, norm):
    x = x.float()
    if norm is None:
        return x
    kind, weight, bias = norm
    if kind == "rms":
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float() + bias.float()


def _turned(x, cos, sin, off, rot, half):
    if rot == 0:
        return x
    part = x[..., off:off + rot]
    if half:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([x[..., :off], turned, x[..., off + rot:]], -1)


def _plain_heads(st):
    """The queries and the keys of norm and append: normed, then turned."""
    angle = (st["positions"].double()[:, None] * _inv_freq(st["scheme"], st["rot"], st["q"].device))[:, None]
    cos, sin = (angle.cos() * st["scheme"]["mscale"]).float(), (angle.sin() * st["scheme"]["mscale"]).float()
    how = (cos, sin, st["off"], st["rot"], st["half"])
    q = _turned(_normed(st["q"], st["q_norm"]), *how).to(st["q"].dtype)
    if st["k"] is None:
        return q, None
    return q, _turned(_normed(st["k"], st["k_norm"]), *how).to(st["k"].dtype)


def _plain_norm(st):
    q, k = _plain_heads(st)
    if k is None:
        return [q]
    if st["rows"] is None:
        return [q, k]
    st["k_out"][st["rows"]] = k
    return [q, st["k_out"]]


def _plain_append(st):
    q, k = _plain_heads(st)
    rows = st["rows"][st["skip"]:]  # padding tokens come first
    st["k_cache"][rows // BLOCK, rows % BLOCK] = k[st["skip"]:]
    st["v_cache"][rows // BLOCK, rows % BLOCK] = st["v"][st["skip"]:]
    return [q, st["k_cache"], st["v_cache"]]


def _plain_attention(st):
    q, H, Hkv = st["q"], st["q"].shape[1], st["k"].shape[-2]
    paged, dev = st["op"] == "paged", st["q"].device
    T, Lq, L = q.shape[0], st["max_q"], st["max_k"]
    i, j = torch.arange(Lq, device=dev), torch.arange(L, device=dev)
    if paged:
        start = torch.arange(0, T, st["S1"], device=dev)
        new = st["q_lens"] if st["q_lens"] is not None else torch.full_like(st["act_seqs"], st["S1"])
    else:
        start, new = st["cu_q"][:-1].long(), st["cu_q"].diff()
    B = new.numel()
    if st["block_table"] is not None:
        act = st["act_seqs"]
        page = st["block_table"].clamp(min=0).long()[:, j // BLOCK]
        k, v = st["k"][page, j % BLOCK].float(), st["v"][page, j % BLOCK].float()
    else:
        act = new
        at = (start[:, None] + j).clamp(max=T - 1)
        k, v = st["k"][at].float(), st["v"][at].float()
    # padded queries [B, Hkv, G * Lq, D] against keys [B, Hkv, D, L]
    rows = (start[:, None] + i).clamp(max=T - 1)
    x = q[rows].float().unflatten(2, (Hkv, H // Hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    z = torch.matmul(x, k.permute(0, 2, 3, 1)).mul_(st["scale"]).unflatten(2, (-1, Lq))
    seen = (j < act[:, None])[:, None] & (i < new[:, None])[:, :, None]
    if st["causal"]:
        seen = seen & (j <= (act - new)[:, None, None] + i[:, None])
    z.masked_fill_(~seen[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(m.masked_fill(m == -math.inf, 0)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).unflatten(2, (-1, Lq)) / l.masked_fill(l == 0, 1)
    lse = (m + l.log()).squeeze(-1)
    o, lse = o.permute(0, 3, 1, 2, 4).flatten(2, 3), lse.permute(0, 3, 1, 2).flatten(2, 3)
    if paged:
        return o.flatten(0, 1).to(q.dtype), lse.flatten(0, 1)
    # back to packed rows; those behind the last sequence stay as they were
    t = torch.arange(T, device=dev)
    b = (torch.searchsorted(st["cu_q"], t.to(torch.int32), right=True) - 1).clamp(max=B - 1)
    s = t - start[b]
    live = s < new[b]
    s = s.clamp(max=Lq - 1)
    return (torch.where(live[:, None, None], o[b, s].to(q.dtype), st["out"]), torch.where(live[:, None], lse[b, s], st["lse"]))


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _own(st)
    if st["op"] == "norm":
        return _plain_norm(st)
    if st["op"] == "append":
        return _plain_append(st)
    return _plain_attention(st)


def _own(st):
    import mla_sparse_top_gb300 as mla

    if st["op"] in ("norm", "append"):
        if "params" not in st:  # what a program makes once: the scheme and the norms of a layer
            st["params"] = mla.rope_params(**st["scheme"])
            st["qn"] = None if st["q_norm"] is None else mla.head_norm(*st["q_norm"])
            st["kn"] = None if st.get("k_norm") is None else mla.head_norm(*st["k_norm"])
        how = dict(params=st["params"], rot_dim=st["rot"], half=st["half"], q_norm=st["qn"], k_norm=st["kn"])
        if st["op"] == "norm":
            mla.mla_norm_rope(st["positions"], st["q"], st["k"], rot_off=st["off"], k_rot_off=st["off"], out=st["q_out"],
                              k_out=st.get("k_out"), k_rows=st["rows"], **how)
            return [st["q_out"]] + ([st["k_out"]] if st["k"] is not None else [])
        mla.mla_kv_append(st["positions"], st["rows"], st["k"], st["v"], st["k_cache"], st["v_cache"], q=st["q"],
                          q_out=st["q_out"], **how)
        return [st["q_out"], st["k_cache"], st["v_cache"]]
    if st["op"] == "prompt":
        if "dims" not in st:
            st["dims"] = mla.prompt_dims(st["q"], st["k"], st["v"], st["cu_q"], block_table=st["block_table"],
                                         causal=st["causal"])
            st["workspace"] = torch.empty(mla.mla_prompt_workspace_bytes(st["dims"]), dtype=torch.uint8, device="cuda")
        return mla.mla_prompt_attn_fwd(st["q"], st["k"], st["v"], st["cu_q"], st["out"], st["lse"], st["workspace"],
                                       block_table=st["block_table"], act_seqs=st.get("act_seqs"),
                                       softmax_scale=st["scale"], dims=st["dims"])
    if "dims" not in st:
        st["dims"] = mla.paged_dims(st["q"], st["k"], st["v"], st["block_table"], S1=st["S1"])
        st["workspace"] = torch.empty(mla.mla_paged_workspace_bytes(st["dims"]), dtype=torch.uint8, device="cuda")
    return mla.mla_paged_attn_fwd(st["q"], st["k"], st["v"], st["block_table"], st["act_seqs"], st["out"], st["lse"],
                                  st["workspace"], q_lens=st["q_lens"], softmax_scale=st["scale"], dims=st["dims"])


# ------------------------------------------------------------------ what a pass cannot do without
def _weights(kind, D, item):
    return 0 if kind == "none" else D * item if kind == "rms" else 8 * D


def work(case):
    item = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "norm":
        T, heads = case["T"], case["H"] + case["K"]
        size = 4 * T + 2 * T * item * heads * case["D"] + (8 * T if case["rows"] else 0)
        size += _weights(case["q_norm"], case["D"], item) + (_weights(case["k_norm"], case["D"], item) if case["K"] else 0)
        normed = (case["H"] if case["q_norm"] != "none" else 0) + case["K"]
        return dict(bytes=size, flops=T * (3 * case["rot"] * heads + 4 * case["D"] * normed))
    if case["op"] == "append":
        T, H, Hkv, D = case["T"], case["H"], case["Hkv"], case["D"]
        live = T - case["skip"]
        size = 12 * T + 4 * T * H * D + 4 * live * Hkv * (D + case["Dv"])
        size += _weights(case["q_norm"], D, item) + _weights(case["k_norm"], D, item)
        normed = (H if case["q_norm"] != "none" else 0) + (Hkv if case["k_norm"] != "none" else 0)
        return dict(bytes=size, flops=T * (3 * case["rot"] * (H + Hkv) + 4 * D * normed))
    new, act = _lengths(case)
    H, Hkv, D, Dv = case["H"], case["Hkv"], case["D"], case["Dv"]
    T = case["B"] * case["S1"] if case["op"] == "paged" else sum(new)
    size = sum(a for n, a in zip(new, act) if n) * Hkv * (D + Dv) * item + T * H * ((D + Dv) * item + 4)
    if case["op"] == "paged" or case["causal"]:
        pairs = sum(n * (a - n) + n * (n + 1) // 2 for n, a in zip(new, act))
    else:
        pairs = sum(n * a for n, a in zip(new, act))
    return dict(bytes=size, flops=2 * H * pairs * (D + Dv))


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_angles(case, positions):
    """Unit complex numbers of each token and pair, the frequencies one by one from their definition."""
    sch, rot = _scheme(case), case["rot"]
    base = sch["theta"]
    if sch["scaling"] == "ntk":
        base *= sch["factor"] ** (rot / max(rot - 2, 1))
    freq = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if sch["scaling"] == "linear":
            f /= sch["factor"]
        if sch["scaling"] == "yarn":
            edge = [rot * math.log(sch["orig_positions"] / (b * 2 * math.pi)) / (2 * math.log(base))
                    for b in (sch["beta_fast"], sch["beta_slow"])]
            first, last = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            mix = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            f = (1 - mix) * f + mix * f / sch["factor"]
        freq.append(f)
    ang = np.outer(positions.cpu().numpy().astype(np.float64), np.array(freq))
    return torch.from_numpy(np.exp(1j * ang) * sch["mscale"]).cuda()[:, None]


def _exact_heads(x, norm, unit, off, rot, half):
    y = x.double().clone()
    if norm is not None:
        if norm[0] == "layer":
            y -= y.sum(-1, keepdim=True) / y.shape[-1]
        y /= ((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + 1e-6).sqrt()
        y *= norm[1].double()
        if norm[2] is not None:
            y += norm[2].double()
    if rot:
        first = slice(off, off + rot // 2) if half else slice(off, off + rot, 2)
        second = slice(off + rot // 2, off + rot) if half else slice(off + 1, off + rot, 2)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * unit
        y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_norm(case, seed):
    st = _prepare_norm(case, seed)
    unit = _exact_angles(case, st["positions"]) if case["rot"] else None
    how = (unit, case["off"], case["rot"], case["half"])
    got = [_exact_heads(st["q"], st["q_norm"], *how)]
    if case["K"]:
        k = _exact_heads(st["k"], st["k_norm"], *how)
        if case["rows"]:
            whole = torch.zeros(st["k_out"].shape, dtype=torch.float64, device="cuda")
            whole[st["rows"]] = k
            k = whole
        got.append(k)
    return got


def _exact_append(case, seed):
    st = _prepare_append(case, seed)
    unit = _exact_angles(case, st["positions"]) if case["rot"] else None
    how = (unit, 0, case["rot"], case["half"])
    got = [_exact_heads(st["q"], st["q_norm"], *how)]
    rows = st["rows"][case["skip"]:]
    for cache, x in ((st["k_cache"], _exact_heads(st["k"], st["k_norm"], *how)), (st["v_cache"], st["v"].double())):
        whole = torch.zeros((cache.shape[0] * BLOCK,) + cache.shape[2:], dtype=torch.float64, device="cuda")
        whole[rows] = x[case["skip"]:]
        got.append(whole.view(cache.shape))
    return got


def _exact_attention(case, seed):
    new, act = _lengths(case)
    H, Hkv, D, Dv = case["H"], case["Hkv"], case["D"], case["Dv"]
    if 2 * H * sum(n * a for n, a in zip(new, act)) * (D + Dv) > 8e12:
        return None
    st = _prepare_attention(case, seed)
    paged, G = case["op"] == "paged", H // Hkv
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf if paged else 0.0, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, a) in enumerate(zip(new, act)):
        first = b * case["S1"] if paged else at
        if n == 0:
            continue
        if st["block_table"] is not None:
            pages = st["block_table"][b, :-(-a // BLOCK)].long()
            k, v = st["k"][pages].flatten(0, 1)[:a], st["v"][pages].flatten(0, 1)[:a]
        else:
            k, v = st["k"][at:at + n], st["v"][at:at + n]
        at += n
        step = max(1, (1 << 27) // (a * G))
        for h in range(Hkv):
            kh, vh = k[:, h].double(), v[:, h].double()
            for s in range(0, n, step):
                e = min(n, s + step)
                # a causal block of queries needs no keys behind its last
                end = a - n + e if st["causal"] else a
                z = torch.einsum("sgd,ad->sga", st["q"][first + s:first + e, h * G:(h + 1) * G].double(), kh[:end]) * st["scale"]
                if st["causal"]:
                    pos = torch.arange(a - n + s, a - n + e, device="cuda")
                    z.masked_fill_((torch.arange(end, device="cuda") > pos[:, None])[:, None], -math.inf)
                w = torch.logsumexp(z, -1)
                lse[first + s:first + e, h * G:(h + 1) * G] = w
                out[first + s:first + e, h * G:(h + 1) * G] = torch.einsum("sga,ad->sgd", z.sub_(w[..., None]).exp_(), vh[:end])
    return [out, lse]


def exact(case, seed):
    if case["op"] == "norm":
        return _exact_norm(case, seed)
    if case["op"] == "append":
        return _exact_append(case, seed)
    return _exact_attention(case, seed)
