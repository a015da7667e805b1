"""The operators of a drafted decode step, as cases to measure: rotary positions, the page plan (block tables and
slot maps from request lengths) and attention of a tree of drafted tokens over the paged cache.

`run` computes the plain form in elementary torch operations, or, where `own` is true, makes the calls that a user
makes of the library. Layouts are those of the library: a cache row is a 512-wide latent (bf16, or INT8 with one
fp32 scale per 128 values) and a 64-wide bf16 rope part, pages are blocks of 128 rows.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
LATENT, ROPE = 512, 64


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request with a small draft and few heads: latency
        dict(name="tree_one_request", op="tree", B=1, S1=8, H=16, lo=1000, hi=1000, int8=False, tree=True, ragged=False),
        # a decode batch without drafts: single tokens, every length another, the causal form
        dict(name="chain_single_token", op="tree", B=64, S1=1, H=128, lo=100, hi=8192, int8=False, tree=False, ragged=False),
        # the ordinary drafted decode step: 64 sequences of about 8192 positions, eight drafted tokens each
        dict(name="tree_decode", op="tree", B=64, S1=8, H=128, lo=8192, hi=8192, int8=False, tree=True, ragged=False),
        # an INT8 cache, lengths from 500 to 20000, drafts of unequal size with padding rows
        dict(name="tree_ragged_int8", op="tree", B=13, S1=17, H=128, lo=500, hi=20000, int8=True, tree=True, ragged=True),
        # one long document with a large draft: the largest call
        dict(name="tree_long_context", op="tree", B=1, S1=64, H=128, lo=131072, hi=131072, int8=False, tree=True, ragged=False),
        # the step's plan for 64 sequences with a drafted tree each: latency
        dict(name="plan_tree_step", op="plan", B=64, S1=8, lo=100, hi=8192, new=8, tree=True, packed=False),
        # admission of 256 prompts of 1 to 4096 tokens, packed one behind the other
        dict(name="plan_packed_prompts", op="plan", B=256, S1=0, lo=1, hi=65, new=4096, tree=False, packed=True),
        # a large decode batch with chains of up to five new tokens
        dict(name="plan_large_batch", op="plan", B=4001, S1=5, lo=1, hi=16384, new=5, tree=False, packed=False),
        # indexer queries and index keys of a decode step: first half of the head, half layout, long-context scaling,
        # the keys written to their cache rows
        dict(name="rope_index_decode", op="rope", T=128, H=64, D=128, off=0, rot=64, half=True, K=128, koff=0,
             rows=True, dtype="bf16", scaling="yarn", factor=40.0, maxpos=163840, pad=0, inverse=False),
        # attention queries (last 64 of 192) and the shared rope key of a prompt chunk
        dict(name="rope_prompt", op="rope", T=8192, H=128, D=192, off=128, rot=64, half=False, K=64, koff=0,
             rows=False, dtype="bf16", scaling="none", factor=1.0, maxpos=8192, pad=0, inverse=False),
        # the way back (the gradient of the rotation) on odd sizes and padded strides, far positions
        dict(name="rope_inverse_odd", op="rope", T=4099, H=17, D=107, off=7, rot=36, half=True, K=0, koff=0,
             rows=False, dtype="fp32", scaling="linear", factor=8.0, maxpos=1 << 20, pad=5, inverse=True),
        # cosines and sines for the prolog, one row per token
        dict(name="rope_table", op="table", T=65536, rot=64, scaling="yarn", factor=40.0, maxpos=163840),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "plan", "rope", "rope", "table"])
    if op == "tree":
        H = rng.choice([1, 5, 16, 24, 64, 100, 128, 128])
        S1 = _log(rng, 1, 100)
        B = _log(rng, 1, 96)
        hi = _log(rng, 1, 60000)
        while B * S1 * H * hi > (1 << 29) or B * S1 * H * 1088 > (1 << 28) or B * hi > (1 << 20):
            B, S1, hi = max(1, B // 2), max(1, S1 * 2 // 3), max(1, hi * 2 // 3)
        return dict(op="tree", B=B, S1=S1, H=H, lo=rng.choice([0, 1 + hi // 40, hi]), hi=hi, int8=rng.random() < 0.4,
                    tree=rng.random() < 0.7, ragged=rng.random() < 0.5)
    if op == "plan":
        if rng.random() < 0.4:
            return dict(op="plan", B=_log(rng, 1, 300), S1=0, lo=0, hi=_log(rng, 1, 5000), new=_log(rng, 1, 4096),
                        tree=False, packed=True)
        S1 = _log(rng, 1, 64)
        return dict(op="plan", B=_log(rng, 1, 4000 // S1 + 1), S1=S1, lo=0, hi=_log(rng, 1, 30000), new=S1,
                    tree=rng.random() < 0.6, packed=False)
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 40.0])
    maxpos = _log(rng, 100, 1 << 20)
    if op == "table":
        return dict(op="table", T=_log(rng, 1, 65536), rot=2 * rng.randint(1, 64), scaling=scaling, factor=factor,
                    maxpos=maxpos)
    rot = rng.choice([64, 64, 128, 2 * rng.randint(1, 100)])
    off = rng.choice([0, 0, 64, rng.randint(0, 130)])
    D = off + rot + rng.choice([0, 0, 64, rng.randint(0, 70)])
    T, H = _log(rng, 1, 20000), rng.choice([1, 3, 16, 64, 128])
    while T * H * D > (1 << 27):
        T = T // 2
    K = rng.choice([0, rot, rot + 8 * rng.randint(0, 9)])
    return dict(op="rope", T=T, H=H, D=D, off=off, rot=rot, half=rng.random() < 0.5, K=K, koff=K - rot if K else 0,
                rows=K > 0 and rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), scaling=scaling,
                factor=factor, maxpos=maxpos, pad=rng.choice([0, 0, 8, 3]), inverse=rng.random() < 0.3)


def _spread(n, lo, hi, turn=0.6180339887498949):
    """n lengths between lo and hi, even in their logarithm, in no order (the same ones for every seed)."""
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [max(lo, min(hi, int(round(math.exp(a + (b - a) * ((i + 1) * turn % 1.0)) - 1)))) for i in range(n)]


def _drafts(case):
    """Drafted tokens of each sequence."""
    if not case["ragged"]:
        return [case["S1"]] * case["B"]
    return [int(case["S1"] * (((i + 1) * 0.7548776662466927) % 1.0) + 0.5) for i in range(case["B"])]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _randint(g, lo, hi, shape, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int64).to(dtype)


def _parents(g, B, S1):
    """parent[b, s] in [-1, s): token s hangs below an earlier one, or below the context."""
    s = torch.arange(S1, device="cuda")
    u = torch.rand((B, S1), generator=g, device="cuda")
    return ((u * (s + 1)).floor().to(torch.int32) - 1).clamp_(max=S1 - 2).contiguous()


def _closure(parents):
    """[B, S1, S1]: which drafted tokens are ancestors of s or s itself. The parent matrix is doubled until every path is in it."""
    B, S1 = parents.shape
    s = torch.arange(S1, device=parents.device)
    r = ((parents[:, :, None] == s) & (s < s[:, None]) | (s == s[:, None])).float()
    for _ in range(max(1, (S1 - 1).bit_length())):
        r = (torch.matmul(r, r) > 0).float()
    return r > 0


def _words(bits):
    """[..., S1] truth values as [..., ceil(S1 / 64)] int64 words, bit j % 64 of word j / 64."""
    S1 = bits.shape[-1]
    n = -(-S1 // 64)
    b = torch.nn.functional.pad(bits, (0, 64 * n - S1)).view(*bits.shape[:-1], n, 64).to(torch.int64)
    return (b << torch.arange(64, device=bits.device)).sum(-1)


def _scheme(case):
    """(theta, scaling, factor, original positions, magnitude): the frequency scheme that a model's configuration gives."""
    yarn = case["scaling"] == "yarn"
    return dict(theta=10000.0, scaling=case["scaling"], factor=case["factor"], orig_positions=4096,
                beta_fast=32.0, beta_slow=1.0, mscale=0.1 * math.log(case["factor"]) + 1.0 if yarn else 1.0)


def _prepare_tree(case, seed):
    g = _gen(seed)
    B, S1, H = case["B"], case["S1"], case["H"]
    drafts = _drafts(case)
    act = [c + n for c, n in zip(_spread(B, case["lo"], case["hi"]), drafts)]
    blocks = [-(-a // BLOCK) for a in act]
    W, used = max(1, max(blocks)), max(1, sum(blocks))
    table = torch.full((B, W), -1, dtype=torch.int32)
    perm = torch.randperm(used, generator=torch.Generator().manual_seed(int(seed))).to(torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    rows = used * BLOCK
    st = dict(op="tree", S1=S1, block_table=table.cuda(), act_seqs=_ints(act),
              tree_lens=_ints(drafts) if case["ragged"] else None, tree_mask=None)
    if case["tree"]:
        bits = _closure(_parents(g, B, S1))
        st["tree_mask"] = _words(bits).contiguous()
        st["bits"] = bits
    if case["int8"]:
        st["kv_nope"] = _randint(g, -127, 128, (rows, LATENT), torch.int8)
        st["kv_scales"] = (torch.rand((rows, LATENT // 128), generator=g, device="cuda") + 0.5) / 64
    else:
        st["kv_nope"] = torch.randn((rows, LATENT), generator=g, device="cuda", dtype=torch.bfloat16)
        st["kv_scales"] = None
    st["kv_rope"] = torch.randn((rows, ROPE), generator=g, device="cuda", dtype=torch.bfloat16)
    st["q_nope"] = torch.randn((B * S1, H, LATENT), generator=g, device="cuda", dtype=torch.bfloat16)
    st["q_rope"] = torch.randn((B * S1, H, ROPE), generator=g, device="cuda", dtype=torch.bfloat16)
    st["scale"] = (LATENT + ROPE) ** -0.5
    return st


def _new_lens(case):
    if case["packed"]:
        return [max(1, n) for n in _spread(case["B"], 1, case["new"], 0.7548776662466927)]
    return [1 + (7 * i + 3) % case["S1"] for i in range(case["B"])]


def _prepare_plan(case, seed):
    g = _gen(seed)
    B, S1 = case["B"], case["S1"]
    ctx, new = _spread(B, case["lo"], case["hi"]), _new_lens(case)
    have = [-(-c // BLOCK) for c in ctx]
    need = [-(-(c + n) // BLOCK) - h for c, n, h in zip(ctx, new, have)]
    W = max(1, max(h + n for h, n in zip(have, need)))
    num_blocks = sum(have) + sum(need) + 100
    perm = torch.randperm(num_blocks, generator=torch.Generator().manual_seed(int(seed))).to(torch.int32)
    start = torch.tensor([0] + have, dtype=torch.int64).cumsum(0)[:B, None]
    w = torch.arange(W)[None]
    mine = w < torch.tensor(have)[:, None]
    table = torch.where(mine, perm[(start + w).clamp(max=num_blocks - 1)], torch.full((B, W), -1, dtype=torch.int32))
    T = sum(new) + 37 if case["packed"] else B * S1  # packed: a capacity, with rows left over
    return dict(op="plan", S1=S1, T=T, num_blocks=num_blocks, ctx_lens=_ints(ctx), new_lens=_ints(new),
                free_blocks=perm[sum(have):].cuda(), block_table=table.cuda(),
                parents=_parents(g, B, S1) if case["tree"] else None)


_TYPES = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)


def _strided(g, T, H, D, pad, dtype):
    return torch.randn((T, H, D + pad), generator=g, device="cuda", dtype=torch.float32).to(dtype)[:, :, :D]


def _prepare_rope(case, seed):
    g = _gen(seed)
    T, dtype = case["T"], _TYPES[case["dtype"]]
    st = dict(op="rope", rot=case["rot"], off=case["off"], koff=case["koff"], half=case["half"],
              inverse=case["inverse"], scheme=_scheme(case), positions=_randint(g, 0, case["maxpos"], (T,)),
              q=_strided(g, T, case["H"], case["D"], case["pad"], dtype), k=None, rows=None)
    st["q_out"] = torch.zeros_like(st["q"])
    if case["K"]:
        st["k"] = _strided(g, T, 1, case["K"], case["pad"], dtype)
        n = 2 * T if case["rows"] else T
        st["k_out"] = torch.zeros((n, 1, case["K"]), device="cuda", dtype=dtype)
        if case["rows"]:  # each key's row of the index-key cache
            st["rows"] = torch.randperm(n, generator=g, device="cuda")[:T].contiguous()
    return st


def prepare(case, seed):
    if case["op"] == "tree":
        return _prepare_tree(case, seed)
    if case["op"] == "plan":
        return _prepare_plan(case, seed)
    if case["op"] == "rope":
        return _prepare_rope(case, seed)
    g = _gen(seed)
    T, r = case["T"], case["rot"] // 2
    return dict(op="table", rot=case["rot"], scheme=_scheme(case), positions=_randint(g, 0, case["maxpos"], (T,)),
                cos=torch.empty((T, r), device="cuda"), sin=torch.empty((T, r), device="cuda"))


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
        at = [rot * math.log(scheme["orig_positions"] / (2 * math.pi * beta)) / (2 * math.log(theta))
              for beta in (scheme["beta_fast"], scheme["beta_slow"])]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
    return f


def _cos_sin(positions, scheme, rot):
    a = positions.double()[:, None] * _inv_freq(scheme, rot, positions.device)
    return (a.cos() * scheme["mscale"]).float(), (a.sin() * scheme["mscale"]).float()


def _rotate(x, cos, sin, off, rot, half):
    x = x.float()
    part = x[..., off:off + rot]
    cos, sin = cos[:, None], sin[:, None]
    if half:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([x[..., :off], turned, x[..., off + rot:]], -1)


def _plain_rope(st):
    cos, sin = _cos_sin(st["positions"], st["scheme"], st["rot"])
    sin = -sin if st["inverse"] else sin
    out = [_rotate(st["q"], cos, sin, st["off"], st["rot"], st["half"]).to(st["q"].dtype)]
    if st["k"] is not None:
        k = _rotate(st["k"], cos, sin, st["koff"], st["rot"], st["half"]).to(st["k"].dtype)
        if st["rows"] is None:
            out.append(k)
        else:
            st["k_out"][st["rows"]] = k
            out.append(st["k_out"])
    return out


def _plain_plan(st):
    S1, nf = st["S1"], st["free_blocks"].numel()
    ctx, new = st["ctx_lens"], st["new_lens"]
    act = ctx + new
    have, total = (ctx + BLOCK - 1) // BLOCK, (act + BLOCK - 1) // BLOCK
    need = total - have
    off = need.cumsum(0) - need
    w = torch.arange(st["block_table"].shape[1], device=ctx.device)[None]
    fresh = (w >= have[:, None]) & (w < total[:, None])
    pick = (off[:, None] + w - have[:, None]).clamp(0, nf - 1)
    table = torch.where(fresh, st["free_blocks"][pick], st["block_table"])
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0)).to(torch.int32)
    if S1:
        s = torch.arange(S1, device=ctx.device, dtype=torch.int32)[None]
        seq = torch.arange(ctx.numel(), device=ctx.device)[:, None].expand(-1, S1)
        valid = s < new[:, None]
        slot = ctx[:, None] + s
        depth = s
    else:
        t = torch.arange(st["T"], device=ctx.device, dtype=torch.int32)
        seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=ctx.numel() - 1)
        valid = t < cu[-1]
        depth = t - cu[seq]
        slot = ctx[seq] + depth
    rows = table[seq, (slot // BLOCK).clamp(0, table.shape[1] - 1).long()].long() * BLOCK + slot % BLOCK
    out = dict(block_table=table, act_seqs=act, cu_seqs=cu, num_taken=need.sum().to(torch.int32).view(1),
               cache_index=torch.where(valid, rows, -1).view(-1),
               seq_ids=torch.where(valid, seq, -1).to(torch.int32).view(-1))
    if st["parents"] is not None:
        up = _closure(st["parents"]) & valid[:, :, None]
        depth = up.sum(-1).to(torch.int32) - 1
        out["tree_mask"] = _words(up).view(-1, -(-S1 // 64))
    pos = ctx[:, None] + depth if S1 else ctx[seq] + depth
    out["positions"] = torch.where(valid, pos, 0).to(torch.int32).view(-1)
    return out


def _plain_tree(st):
    table, act, S1 = st["block_table"], st["act_seqs"], st["S1"]
    B, L = table.shape[0], table.shape[1] * BLOCK
    H = st["q_nope"].shape[1]
    j = torch.arange(L, device=table.device)
    rows = table.clamp(min=0).long()[:, j // BLOCK] * BLOCK + j % BLOCK
    nope = st["kv_nope"][rows].float()
    if st["kv_scales"] is not None:
        nope = (nope.view(B, L, 4, 128) * st["kv_scales"][rows][..., None]).to(torch.bfloat16).float().view(B, L, LATENT)
    rope = st["kv_rope"][rows].float()
    drafts = st["tree_lens"] if st["tree_lens"] is not None else torch.full_like(act, S1)
    ctx = act - drafts
    s = torch.arange(S1, device=table.device)
    if st["tree_mask"] is not None:
        words = st["tree_mask"].view(B, S1, -1)
        sees = (words[..., s // 64] >> (s % 64) & 1).bool()
    else:
        sees = (s <= s[:, None])[None].expand(B, -1, -1)
    sees = sees & (s[None, None, :] < drafts[:, None, None])
    k = j[None] - ctx[:, None]  # which drafted token a position holds
    drafted = torch.gather(sees, 2, k.clamp(0, S1 - 1)[:, None, :].expand(-1, S1, -1))
    visible = torch.where((k >= 0)[:, None], drafted, True) & (j[None] < act[:, None])[:, None]
    visible = visible & (s[None] < drafts[:, None])[:, :, None]  # [B, S1, L]
    q = torch.cat([st["q_nope"], st["q_rope"]], -1).float().view(B, S1 * H, LATENT + ROPE)
    z = torch.matmul(q, torch.cat([nope, rope], -1).transpose(1, 2)).mul_(st["scale"]).view(B, S1, H, L)
    z.masked_fill_(~visible[:, :, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(m.masked_fill(m == -math.inf, 0)).exp_()
    l = p.sum(-1, keepdim=True)
    dead = torch.arange(L, device=table.device)[None] >= act[:, None]
    v = nope.masked_fill_(dead[..., None], 0)
    o = torch.matmul(p.view(B, S1 * H, L), v).view(B, S1, H, LATENT) / l.masked_fill(l == 0, 1)
    lse = (m + l.log()).view(B * S1, H)
    return o.to(torch.bfloat16).view(B * S1, H, LATENT), lse


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _own(st)
    if st["op"] == "tree":
        return _plain_tree(st)
    if st["op"] == "plan":
        return _plain_plan(st)
    if st["op"] == "rope":
        return _plain_rope(st)
    return list(_cos_sin(st["positions"], st["scheme"], st["rot"]))


def _own(st):
    import mla_sparse_top_gb300 as mla

    if st["op"] == "tree":
        if "out" not in st:  # a program keeps its outputs and its workspace from step to step
            st["out"] = torch.empty_like(st["q_nope"])
            st["lse"] = torch.empty(st["q_nope"].shape[:2], dtype=torch.float32, device="cuda")
            st["dims"] = mla.tree_dims(st["q_nope"], st["kv_nope"], st["block_table"], S1=st["S1"])
            st["workspace"] = torch.empty(mla.mla_tree_workspace_bytes(st["dims"]), dtype=torch.uint8, device="cuda")
        return mla.mla_tree_attn_fwd(st["q_nope"], st["q_rope"], st["kv_nope"], st["kv_rope"], st["kv_scales"],
                                     st["block_table"], st["act_seqs"], st["out"], st["lse"], st["workspace"],
                                     tree_lens=st["tree_lens"], tree_mask=st["tree_mask"], softmax_scale=st["scale"],
                                     dims=st["dims"])
    if st["op"] == "plan":
        if "outputs" not in st:
            B, T, S1 = st["ctx_lens"].numel(), st["T"], st["S1"]
            new = lambda shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
            st["outputs"] = dict(act_seqs=new(B), cu_seqs=new(B + 1), num_taken=new(1), positions=new(T),
                                 seq_ids=new(T), cache_index=new(T, torch.int64))
            if st["parents"] is not None:
                st["outputs"]["tree_mask"] = new((T, -(-S1 // 64)), torch.int64)
        mla.mla_page_plan(st["ctx_lens"], st["new_lens"], st["free_blocks"], st["block_table"], S1=st["S1"],
                          num_blocks=st["num_blocks"], parents=st["parents"], **st["outputs"])
        return dict(st["outputs"], block_table=st["block_table"])
    if "params" not in st:
        st["params"] = mla.rope_params(**st["scheme"])
    if st["op"] == "table":
        mla.mla_rope_table(st["positions"], st["cos"], st["sin"], params=st["params"])
        return [st["cos"], st["sin"]]
    mla.mla_rope_apply(st["positions"], st["q"], st["k"], params=st["params"], rot_dim=st["rot"], rot_off=st["off"],
                       k_rot_off=st["koff"], half=st["half"], inverse=st["inverse"], out=st["q_out"],
                       k_out=st.get("k_out"), k_rows=st["rows"])
    return [st["q_out"]] + ([st["k_out"]] if st["k"] is not None else [])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "tree":
        drafts, ctx = _drafts(case), _spread(case["B"], case["lo"], case["hi"])
        row = (LATENT + 16 if case["int8"] else 2 * LATENT) + 2 * ROPE
        T = case["B"] * case["S1"]
        words = 8 * -(-case["S1"] // 64) if case["tree"] else 0
        size = sum((c + n) * row for c, n in zip(ctx, drafts)) + T * words
        size += T * case["H"] * (2 * (LATENT + ROPE) + 2 * LATENT + 4)
        pairs = sum(n * (c + (n + 1) / 2) for c, n in zip(ctx, drafts))
        return dict(bytes=size, flops=2 * case["H"] * pairs * (2 * LATENT + ROPE))
    if case["op"] == "plan":
        ctx, new = _spread(case["B"], case["lo"], case["hi"]), _new_lens(case)
        need = sum(-(-(c + n) // BLOCK) - -(-c // BLOCK) for c, n in zip(ctx, new))
        T = sum(new) + 37 if case["packed"] else case["B"] * case["S1"]
        size = 16 * case["B"] + 8 * need + T * 16
        if case["tree"]:
            size += T * (4 + 8 * -(-case["S1"] // 64))
        return dict(bytes=size, flops=0)
    if case["op"] == "table":
        return dict(bytes=case["T"] * (4 + 4 * case["rot"]), flops=10 * case["T"] * case["rot"])
    T, item = case["T"], 4 if case["dtype"] == "fp32" else 2
    # the keys' output is compared whole, but only the written rows cost anything
    size = T * 4 + 2 * T * item * (case["H"] * case["D"] + case["K"]) + (8 * T if case["rows"] else 0)
    return dict(bytes=size, flops=3 * T * case["rot"] * (case["H"] + (1 if case["K"] else 0)))


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_tree(case, seed):
    st = _prepare_tree(case, seed)
    B, S1, H = case["B"], case["S1"], case["H"]
    out = torch.zeros((B, S1, H, LATENT), dtype=torch.float64, device="cuda")
    lse = torch.full((B, S1, H), -math.inf, dtype=torch.float64, device="cuda")
    drafts, act = _drafts(case), st["act_seqs"].tolist()
    for b in range(B):
        n, a = drafts[b], act[b]
        if n == 0 or a == 0:
            continue
        pages = st["block_table"][b, :-(-a // BLOCK)].long()
        rows = (pages[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten()[:a]
        c = st["kv_nope"][rows].double()
        if case["int8"]:
            # a cache value is defined as the bf16 nearest to the fp32 product of code and scale
            c = (c.float() * st["kv_scales"][rows].repeat_interleave(128, 1)).to(torch.bfloat16).double()
        r = st["kv_rope"][rows].double()
        step = max(1, (1 << 28) // (a * H))
        for s0 in range(0, n, step):
            for_s = slice(b * S1 + s0, b * S1 + min(n, s0 + step))
            k = for_s.stop - for_s.start
            z = torch.einsum("shd,ad->sha", st["q_nope"][for_s].double(), c)
            z += torch.einsum("shd,ad->sha", st["q_rope"][for_s].double(), r)
            z *= st["scale"]
            if case["tree"]:
                see = st["bits"][b, s0:s0 + k, :n]
            else:
                see = torch.arange(n, device="cuda")[None] <= torch.arange(s0, s0 + k, device="cuda")[:, None]
            z[:, :, a - n:].masked_fill_(~see[:, None], -math.inf)
            e = torch.logsumexp(z, -1)
            lse[b, s0:s0 + k] = e
            out[b, s0:s0 + k] = torch.einsum("sha,ad->shd", z.sub_(e[..., None]).exp_(), c)
            del z
    return [out.view(B * S1, H, LATENT), lse.view(B * S1, H)]


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
    return torch.from_numpy(np.exp(1j * ang) * sch["mscale"]).cuda()


def _exact_rope(case, seed):
    st = _prepare_rope(case, seed)
    unit = _exact_angles(case, st["positions"])[:, None]
    unit = unit.conj() if case["inverse"] else unit

    def turn(x, off):
        y, r = x.double().clone(), case["rot"]
        first = slice(off, off + r // 2) if case["half"] else slice(off, off + r, 2)
        second = slice(off + r // 2, off + r) if case["half"] else slice(off + 1, off + r, 2)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    got = [turn(st["q"], case["off"])]
    if case["K"]:
        k = turn(st["k"], case["koff"])
        if case["rows"]:
            whole = torch.zeros(st["k_out"].shape, dtype=torch.float64, device="cuda")
            whole[st["rows"]] = k
            k = whole
        got.append(k)
    return got


def exact(case, seed):
    if case["op"] == "tree":
        return _exact_tree(case, seed)
    if case["op"] == "plan":
        return None  # whole numbers throughout
    if case["op"] == "rope":
        return _exact_rope(case, seed)
    unit = _exact_angles(case, prepare(case, seed)["positions"])
    return [unit.real.contiguous(), unit.imag.contiguous()]
