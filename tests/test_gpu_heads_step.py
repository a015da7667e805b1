"""One attention layer as it is served: page plan, append of keys and values with norms and rotation, attention of
prompts and then of new tokens over the same pages, every stage against its oracle on what the stage before left."""
import pytest
import torch

from heads_util import TYPES, cache, check_sequence, gather, normal
from test_gpu_heads_prep import check as check_prep, make_norm

pytestmark = pytest.mark.gpu

SCHEME = dict(scaling="yarn", factor=4.0)


class Layer:
    """Heads, pools and tables of one layer; `run` enqueues a step, `check` holds it against the oracles."""

    def __init__(self, B, *, H, Hkv, D, Dv, rot, dtype, layout, kind="rms", blocks=64, W=12, seed=0):
        import mla_sparse_top_gb300 as mla
        self.mla, self.dt, self.B, self.W, self.blocks = mla, TYPES[dtype], B, W, blocks
        self.H, self.Hkv, self.D, self.Dv, self.rot = H, Hkv, D, Dv, rot
        self.gen = torch.Generator().manual_seed(seed)
        self.k = cache(blocks, Hkv, D, layout, self.dt, fill=float("nan"))
        self.v = cache(blocks, Hkv, Dv, layout, self.dt, fill=float("nan"))
        (self.qn, self.q_norm), (self.kn, self.k_norm) = (make_norm(kind, D, self.dt, f, seed=3 + f) for f in (True, False))
        self.params = mla.rope_params(**SCHEME)
        self.table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(blocks, generator=self.gen).to(torch.int32).tolist()
        self.ctx = [0] * B
        self.raw = [([], []) for _ in range(B)]  # keys and values of each sequence as they came in

    def buffers(self, T):
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(T=T, ctx=torch.zeros(self.B, **i32), new=torch.zeros(self.B, **i32),
                    free=torch.zeros(self.blocks, **i32), act=torch.zeros(self.B, **i32), positions=torch.zeros(T, **i32),
                    index=torch.zeros(T, dtype=torch.int64, device="cuda"), cu=torch.zeros(self.B + 1, **i32),
                    qk=torch.zeros((T, self.H + self.Hkv, self.D), dtype=self.dt, device="cuda"),
                    v=torch.zeros((T, self.Hkv, self.Dv), dtype=self.dt, device="cuda"),
                    out=torch.zeros((T, self.H, self.Dv), dtype=self.dt, device="cuda"),
                    lse=torch.zeros((T, self.H), device="cuda"))

    def fill(self, s, new, S1):
        """New tokens, lengths and free pages of a step; padding rows hold NaN."""
        rows = [r for b, n in enumerate(new) for r in range(b * S1, b * S1 + n)] if S1 else list(range(sum(new)))
        s["qk"].fill_(float("nan"))
        s["v"].fill_(float("nan"))
        s["qk"][rows] = normal(self.gen, (len(rows), self.H + self.Hkv, self.D), self.dt)
        s["v"][rows] = normal(self.gen, (len(rows), self.Hkv, self.Dv), self.dt)
        s["q_raw"] = s["qk"][:, :self.H].clone()
        at = 0
        s["rows"] = []
        for b, n in enumerate(new):
            mine = rows[at:at + n]
            s["rows"].append(mine)
            self.raw[b][0].append(s["qk"][mine, self.H:].clone())
            self.raw[b][1].append(s["v"][mine].clone())
            at += n
        s["ctx"].copy_(torch.tensor(self.ctx, dtype=torch.int32))
        s["new"].copy_(torch.tensor(new, dtype=torch.int32))
        need = sum(-(-(c + n) // 128) - -(-c // 128) for c, n in zip(self.ctx, new))
        s["free"].copy_(torch.tensor((self.free + [0] * self.blocks)[:self.blocks], dtype=torch.int32))
        self.free = self.free[need:]
        self.ctx = [c + n for c, n in zip(self.ctx, new)]
        s["out"].fill_(float("nan"))
        s["lse"].fill_(float("nan"))

    def run(self, s, S1, stream=None):
        mla = self.mla
        mla.mla_page_plan(s["ctx"], s["new"], s["free"], self.table, s["act"], s["index"], S1=S1, num_blocks=self.blocks,
                          positions=s["positions"], cu_seqs=s["cu"], stream=stream)
        q, k = s["qk"][:, :self.H], s["qk"][:, self.H:]
        mla.mla_kv_append(s["positions"], s["index"], k, s["v"], self.k, self.v, params=self.params, rot_dim=self.rot,
                          half=True, q=q, q_norm=self.q_norm, k_norm=self.k_norm, stream=stream)
        if S1 == 0:
            dims = mla.prompt_dims(q, self.k, self.v, s["cu"], block_table=self.table)
            if "ws" not in s:
                s["ws"] = torch.empty(mla.mla_prompt_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
            mla.mla_prompt_attn_fwd(q, self.k, self.v, s["cu"], s["out"], s["lse"], s["ws"], block_table=self.table,
                                    act_seqs=s["act"], softmax_scale=self.D ** -0.5, dims=dims, stream=stream)
        else:
            dims = mla.paged_dims(q, self.k, self.v, self.table, S1=S1)
            if "ws" not in s:
                s["ws"] = torch.empty(mla.mla_paged_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
            mla.mla_paged_attn_fwd(q, self.k, self.v, self.table, s["act"], s["out"], s["lse"], s["ws"],
                                   q_lens=s["new"], softmax_scale=self.D ** -0.5, dims=dims, stream=stream)

    def check(self, s, S1):
        mla = self.mla
        torch.cuda.synchronize()
        assert mla.heads_device_status(clear=True) == 0 and mla.page_device_status(clear=True) == 0
        kw = dict(rot_dim=self.rot, rot_off=0, half=True)
        table = self.table.cpu()
        for b, rows in enumerate(s["rows"]):
            L, n = self.ctx[b], len(rows)
            k, v = gather(self.k, table, b, L), gather(self.v, table, b, L)
            if L:
                pos = torch.arange(L, dtype=torch.int32)
                check_prep(k, torch.cat(self.raw[b][0]), pos, self.kn, SCHEME, f"keys {b}", **kw)
                assert torch.equal(v, torch.cat(self.raw[b][1]).cpu())
            if n:
                pos = torch.arange(L - n, L, dtype=torch.int32)
                check_prep(s["qk"][rows, :self.H], s["q_raw"][rows], pos, self.qn, SCHEME, f"queries {b}", **kw)
                check_sequence(s["out"][rows], s["lse"][rows], s["qk"][rows, :self.H], k, v, self.D ** -0.5, True,
                               f"sequence {b}")
        live = sorted(r for rows in s["rows"] for r in rows)
        dead = [r for r in range(s["T"]) if r not in set(live)]
        if S1:  # padding rows see nothing
            assert (s["out"][dead] == 0).all() and torch.isneginf(s["lse"][dead]).all()
        else:   # rows behind the last sequence stay
            assert torch.isnan(s["out"][dead]).all() and torch.isnan(s["lse"][dead]).all()
        # rows of the pools that no token has stay as they were
        used = torch.zeros((self.blocks, 128), dtype=torch.bool)
        for b in range(self.B):
            for p in range(self.ctx[b]):
                used[table[b, p // 128], p % 128] = True
        assert torch.isnan(self.k.cpu()[~used]).all() and torch.isnan(self.v.cpu()[~used]).all()


CASES = [
    dict(H=12, Hkv=4, D=128, Dv=128, rot=128, dtype="bf16", layout="token"),
    dict(H=14, Hkv=2, D=96, Dv=64, rot=64, dtype="fp16", layout="head", kind="layer"),
    dict(H=5, Hkv=5, D=64, Dv=64, rot=32, dtype="bf16", layout="shared"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_prompts_chunks_and_new_tokens(case):
    layer = Layer(3, **case)
    for new in ([130, 40, 0], [300, 1, 257]):  # prompts, then chunks over what their pages hold, rows left over
        s = layer.buffers(570)
        layer.fill(s, new, 0)
        layer.run(s, 0)
        layer.check(s, 0)
    for S1, new in ((1, [1, 1, 1]), (4, [4, 0, 2]), (4, [1, 3, 4])):
        s = layer.buffers(3 * S1)
        layer.fill(s, new, S1)
        layer.run(s, S1)
        layer.check(s, S1)


def test_steps_captured_once_and_replayed():
    """A chunk's step and a decode step, each one graph on another stream, replayed on new lengths and tokens."""
    layer = Layer(3, **CASES[0])
    graphs = {}
    side = torch.cuda.Stream()
    for S1, T in ((0, 400), (3, 9)):
        s = layer.buffers(T)
        warm = Layer(3, **CASES[0])  # the first calls, on pools of their own
        w = warm.buffers(T)
        warm.fill(w, [2, 0, 3], S1)
        warm.run(w, S1)
        warm.check(w, S1)
        s["ws"] = w["ws"]
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            layer.run(s, S1)
        graphs[S1] = (g, s)
    for S1, new in ((0, [200, 129, 1]), (0, [0, 5, 300]), (3, [1, 1, 1]), (3, [3, 0, 2]), (0, [7, 0, 128]), (3, [0, 3, 1])):
        g, s = graphs[S1]
        layer.fill(s, new, S1)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g.replay()
        torch.cuda.current_stream().wait_stream(side)
        layer.check(s, S1)


def test_chunks_write_the_keys_of_the_whole_prompt():
    """A prompt in one call and in chunks over the pages: keys alike to the bit, outputs each within their bound."""
    case = dict(CASES[0], dtype="fp16")
    whole, cut = Layer(1, **case), Layer(1, **case)
    s = whole.buffers(500)
    whole.fill(s, [500], 0)
    whole.run(s, 0)
    whole.check(s, 0)
    x, v = torch.cat([s["q_raw"], whole.raw[0][0][0]], 1), s["v"].clone()
    for a, e in ((0, 1), (1, 128), (128, 300), (300, 499), (499, 500)):
        c = cut.buffers(e - a)
        cut.fill(c, [e - a], 0)
        c["qk"].copy_(x[a:e])
        c["v"].copy_(v[a:e])
        c["q_raw"].copy_(x[a:e, :cut.H])
        cut.raw[0][0][-1].copy_(x[a:e, cut.H:])
        cut.raw[0][1][-1].copy_(v[a:e])
        cut.run(c, 0)
        cut.check(c, 0)
    k1, k2 = gather(whole.k, whole.table.cpu(), 0, 500), gather(cut.k, cut.table.cpu(), 0, 500)
    assert torch.equal(k1, k2)


def test_two_graphs_share_a_workspace():
    """Prompts that are cut, prompts that are not and new tokens, captured with one workspace, replayed in any order."""
    import test_gpu_heads_paged as paged
    import test_gpu_heads_prompt as prompt
    import mla_sparse_top_gb300 as mla
    calls = [(prompt, prompt.make([60, 9], ctx=[20000, 300], paged=True, H=8, Hkv=2, D=128, Dv=128)),
             (prompt, prompt.make([500, 1, 700], H=8, Hkv=2, D=128, Dv=128)),
             (paged, paged.make([5000, 0, 300], H=8, Hkv=2, S1=2)), (paged, paged.make([700] * 40, H=4, Hkv=2, D=64, Dv=64))]
    want = [mod.run(m) for mod, m in calls]
    ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device="cuda")
    graphs = []
    for mod, m in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = mod.run(m, workspace=ws)
        graphs.append((g, out))
    for i in (0, 2, 1, 3, 3, 0, 1, 2, 0):
        g, (out, lse) = graphs[i]
        out.fill_(7.0), lse.fill_(7.0)
        g.replay()
        a, b = want[i]
        live = ~torch.isnan(b) if calls[i][0] is paged else b != 7  # rows behind the last sequence stay
        assert torch.equal(lse[live], b[live]) and torch.equal(out[live], a[live])
    assert mla.heads_device_status(clear=True) == 0


def test_calls_on_two_streams():
    """The same kinds of calls side by side, a workspace each: results to the bit."""
    import test_gpu_heads_prompt as prompt
    import mla_sparse_top_gb300 as mla
    ms = [prompt.make([300, 90], ctx=[9000, 0], paged=True, H=8, Hkv=2, D=128, Dv=128), prompt.make([900, 1100], H=16, Hkv=4, D=64, Dv=64)]
    want = [prompt.run(m) for m in ms]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ms], []
    for _ in range(4):
        for m, s in zip(ms, streams):
            with torch.cuda.stream(s):
                got.append(prompt.run(m))
    torch.cuda.synchronize()
    assert mla.heads_device_status(clear=True) == 0
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
