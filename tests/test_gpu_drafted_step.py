"""A drafted decode step as a user chains the calls: the page plan makes block
tables, slots, positions and tree masks from request lengths; the rotary table
makes the prolog's cosines and sines; the prolog writes the drafts' cache rows
and the absorbed queries; the index keys are rotated into their own paged
cache; attention runs over context and tree.  The whole step is captured once
and replayed on other lengths.  The oracles run the same chain.

Tolerance of the output: that of the prolog-then-attention chain (the chains
differ where the prolog's bf16 roundings do; |gpu - oracle| <= 1e-2 |oracle| +
1e-2 rms(row) at a scale of 0.05 / sqrt(576)), to which the attention adds the
rounding of its weights, 2^-8 sum_p p |v_p| at most."""
import numpy as np
import pytest
import torch

import workloads
from oracle import prolog as P
from oracle import step

pytestmark = pytest.mark.gpu
S1, H, BLOCKS, W = 5, 128, 24, 6
YARN = dict(scaling="yarn", factor=8.0, orig_positions=128)


def lengths(seed):
    rng = np.random.default_rng(seed)
    ctx = np.array([130, 7, 0, 250][seed % 2:][:3] + [int(rng.integers(100, 400))], np.int32)
    new = np.array([5, 3, 5, 1], np.int32)
    parents = (rng.random((4, S1)) * (np.arange(S1) + 1)).astype(np.int32) - 1
    perm = rng.permutation(BLOCKS).astype(np.int32)
    table = np.full((4, W), -1, np.int32)
    at = 0
    for b in range(4):
        n = -(-int(ctx[b]) // 128)
        table[b, :n] = perm[at:at + n]
        at += n
    return ctx, new, parents, table, perm[at:at + 8]


@pytest.mark.parametrize("kv_int8", [False, True])
def test_step_and_its_replay_match_the_oracles(kv_int8):
    import mla_sparse_top_gb300 as mla
    B, T = 4, 4 * S1
    inp = workloads.make_prolog_inputs(T=T, seed=80 + kv_int8, hidden=256, q_lora=128, n_heads=H, num_blocks=BLOCKS,
                                       kv_int8=kv_int8)
    g = torch.Generator().manual_seed(3)
    rows = BLOCKS * 128
    if kv_int8:
        inp["kv_nope"] = torch.randint(-127, 128, (rows, 512), generator=g).to(torch.int8).numpy()
        inp["kv_scales"] = np.full((rows, 4), 1 / 64, np.float32)
    else:
        inp["kv_nope"] = torch.randn((rows, 512), generator=g).bfloat16().view(torch.int16).numpy().view(np.uint16)
    inp["kv_rope"] = torch.randn((rows, 64), generator=g).bfloat16().view(torch.int16).numpy().view(np.uint16)
    scale = 0.05 * 576 ** -0.5
    dev = workloads.prolog_to_device(inp)
    cache0 = [dev[k].clone() for k in ("kv_nope", "kv_rope")] + [dev["kv_scales"].clone() if kv_int8 else None]
    i32 = dict(dtype=torch.int32, device="cuda")
    t32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    ctx, new, parents, table, free = (t32(a) for a in lengths(0))
    act, taken, pos = torch.zeros(B, **i32), torch.zeros(1, **i32), torch.zeros(T, **i32)
    slots, mask = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    cos, sin = torch.zeros((2, T, 32), device="cuda")
    q_nope = torch.zeros((T, H, 512), dtype=torch.bfloat16, device="cuda")
    q_rope = torch.zeros((T, H, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q_nope), torch.zeros((T, H), device="cuda")
    iq = torch.randn((T, 16, 128), generator=g).bfloat16().cuda()
    ik = torch.randn((T, 1, 128), generator=g).bfloat16().cuda()
    iq_out, icache = torch.zeros_like(iq), torch.zeros((rows, 1, 128), dtype=torch.bfloat16, device="cuda")
    par = mla.rope_params(**YARN)
    pws = torch.empty(mla.mla_prolog_workspace_bytes(mla.prolog_dims(dev["x"], dev["wq_a"], dev["wq_b"], dev["kv_nope"])),
                      dtype=torch.uint8, device="cuda")
    dims = mla.tree_dims(q_nope, dev["kv_nope"], table, S1=S1)
    tws = torch.empty(mla.mla_tree_workspace_bytes(dims), dtype=torch.uint8, device="cuda")

    def one_step():
        mla.mla_page_plan(ctx, new, free, table, act, slots, S1=S1, num_blocks=BLOCKS, parents=parents, positions=pos,
                          tree_mask=mask, num_taken=taken)
        mla.mla_rope_table(pos, cos, sin, params=par)
        mla.mla_prolog(dev["x"], dev["wq_a"], dev["gamma_cq"], dev["wq_b"], dev["w_uk"], dev["wkv"], dev["gamma_ckv"],
                       cos, sin, slots, q_nope, q_rope, dev["kv_nope"], dev["kv_rope"], dev["kv_scales"], pws)
        mla.mla_rope_apply(pos, iq, ik, params=par, rot_dim=64, half=True, out=iq_out, k_out=icache, k_rows=slots)
        mla.mla_tree_attn_fwd(q_nope, q_rope, dev["kv_nope"], dev["kv_rope"], dev["kv_scales"], table, act, out, lse,
                              tws, tree_lens=new, tree_mask=mask, softmax_scale=scale, dims=dims)

    def restore(lens):
        for t, a in zip((ctx, new, parents, table), lens[:4]):
            t.copy_(t32(a))
        free.copy_(t32(lens[4]))
        dev["kv_nope"].copy_(cache0[0])
        dev["kv_rope"].copy_(cache0[1])
        if kv_int8:
            dev["kv_scales"].copy_(cache0[2])
        icache.zero_()

    def check(lens):
        c, n, p, tab, fr = lens
        plan = step.page_plan(c, n, fr, tab, S1=S1, T=T, num_blocks=BLOCKS, parents=p)
        np.testing.assert_array_equal(slots.cpu().numpy(), plan["cache_index"])
        np.testing.assert_array_equal(table.cpu().numpy(), plan["block_table"])
        np.testing.assert_array_equal(act.cpu().numpy(), plan["act_seqs"])
        np.testing.assert_array_equal(pos.cpu().numpy(), plan["positions"])
        freqs = step.rope_freqs(64, **YARN)
        ang = plan["positions"][:, None] * freqs
        ref, (kn, kr, ks, bad) = P.forward_with_cache({**inp, "cos": np.cos(ang), "sin": np.sin(ang),
                                                       "cache_index": plan["cache_index"]})
        assert bad == 0
        lat = (kn.astype(np.float32) * np.repeat(ks, 128, 1)) if kv_int8 else P.bf16_to_f64(kn)
        lat = P.round_bf16(lat)
        o, e, mag = step.tree_attention(P.round_bf16(ref["q_nope"]), P.round_bf16(ref["q_rope"]), lat, P.bf16_to_f64(kr),
                                        plan["block_table"], plan["act_seqs"], n, plan["tree_mask"], S1, scale)
        got = out.double().cpu().numpy()
        rms = np.sqrt(np.mean(o ** 2, -1, keepdims=True))
        err = np.abs(got - o)
        assert (err <= 1e-2 * np.abs(o) + 1e-2 * rms + 2.0 ** -8 * mag).all(), float((err / (rms + 1e-30)).max())
        el = lse.double().cpu().numpy()
        assert (np.isneginf(el) == np.isneginf(e)).all()
        np.testing.assert_allclose(el[np.isfinite(e)], e[np.isfinite(e)], rtol=1e-2, atol=1e-2)
        # index keys: only the drafts' rows, rotated (one bf16 rounding, fp32 before it: below one step of bf16)
        written = plan["cache_index"][plan["cache_index"] >= 0]
        k = step.rope_apply(ik.double().cpu().numpy(), plan["positions"], freqs, rot_off=0, half=True)
        kc = icache.double().cpu().numpy()
        np.testing.assert_allclose(kc[written], k[plan["cache_index"] >= 0], rtol=2.0 ** -7, atol=1e-6)
        rest = np.ones(rows, bool)
        rest[written] = False
        assert (kc[rest] == 0).all()

    one_step()
    torch.cuda.synchronize()
    check(lengths(0))
    graph = torch.cuda.CUDAGraph()
    restore(lengths(0))
    with torch.cuda.graph(graph):
        one_step()
    for seed in (0, 1, 2):
        restore(lengths(seed))
        graph.replay()
        torch.cuda.synchronize()
        check(lengths(seed))
    for status in (mla.page_device_status, mla.rope_device_status, mla.prolog_device_status, mla.tree_device_status):
        assert status(clear=True) == 0
