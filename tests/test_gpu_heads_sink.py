"""One key that outweighs all others, whose many small weights still have to count.

Queries are the first unit vector, so a score is its key's first value times the scale, and expected results come
from running sums in fp64.  The sink's own value is 0: out is made of the others alone, whose weights lie between
2^-23 and 2^-31 of the sink's.  Bound of an output as in heads_util.py, but for fp16: the largest weight is at least
2^7 there, so one below the normal range, off by 2^-25 at most, is off by 2^-32 of the largest."""
import pytest
import torch

from heads_util import TYPES, U
import test_gpu_heads_paged as paged
import test_gpu_heads_prompt as prompt

pytestmark = pytest.mark.gpu
GAP = 18.5  # nats from the sink to the middle of the others


def fill(m, b, length, sink):
    """Sequence b's keys and values: the sink at key `sink`, the others random; (length,) scores and (length, Dv) values."""
    gen = torch.Generator().manual_seed(length)
    dt = m["dtype"]
    z = (torch.rand(length, generator=gen) * 5 - 2.5).to(dt)
    z[sink] = GAP
    v = (torch.rand((length, m["Dv"]), generator=gen) + 0.5).to(dt)
    v[sink] = 0
    k = torch.zeros((length, m["D"]), dtype=dt)
    k[:, 0] = z
    if m.get("paged", True):
        for p in range(-(-length // 128)):
            page = m["table_cpu"][b, p].item()
            n = min(128, length - 128 * p)
            m["k"][page, :n] = k[128 * p:128 * p + n, None].cuda()
            m["v"][page, :n] = v[128 * p:128 * p + n, None].cuda()
    else:
        m["k"][:length] = k[:, None].cuda()
        m["v"][:length] = v[:, None].cuda()
    m["q"].zero_()
    m["q"][..., 0] = 1
    return z.double().cuda(), v.double().cuda()


def check(got, lse, z, v, what):
    """n rows, the newest tokens of the keys; every head has the same."""
    n, L = got.shape[0], z.numel()
    w = (z - GAP).exp()
    total, sums = w.cumsum(0)[L - n:], (w[:, None] * v).cumsum(0)[L - n:]
    want = (sums / total[:, None])[:, None]  # values are above 0: their own mass
    info = torch.finfo(got.dtype)
    dz = 2 * U * 192 * GAP + 8 * U * (GAP + 1)
    bound = want * (info.eps / 2 + 2 * dz + 2 * U * (L + 16)) * (1 + 1e-3) + want.clamp(min=info.smallest_normal) * info.eps / 2
    if got.dtype == torch.float16:
        bound = bound + L * v.max() * 2.0 ** -32
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), f"{what}: worst {(err / bound).max().item()}, {got.flatten()[:4].tolist()} for {want.flatten()[:4].tolist()}"
    off = (lse.double() - (GAP + total.log())[:, None]).abs().max().item()
    assert off <= dz + 2 * U * (L + 16) + 4 * U * GAP, f"{what}: lse {off}"


# whole heads (many sequences), cut ones (one), rows of several pipelines, and rows for the prompts' tiles
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B,S1,kw", [(1, 1, dict(H=8, Hkv=1)), (160, 1, dict(H=8, Hkv=8)), (3, 5, dict(H=8, Hkv=1, D=64, Dv=64)),
                                     (2, 3, dict(H=64, Hkv=2, D=192)), (2, 40, dict(H=4, Hkv=1, D=96, Dv=96))])
def test_new_tokens_behind_a_sink(B, S1, kw, dtype):
    length = 3000 if B == 160 else 50000
    m = paged.make([length] * B, S1=S1, dtype=dtype, scale=1.0, **kw)
    sinks = {0: 0, B // 2: 1500, B - 1: length - S1 - 40}
    want = {b: fill(m, b, length, s) for b, s in sinks.items()}
    out, lse = paged.run(m)
    for b, (z, v) in want.items():
        check(out[b * S1:(b + 1) * S1], lse[b * S1:(b + 1) * S1], z, v, f"sequence {b}, sink at {sinks[b]}")
    import mla_sparse_top_gb300 as mla
    assert mla.heads_device_status(clear=True) == 0


# an SM alone, values of up to 64 columns, pairs of SMs; cut and whole
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,length,kw", [(20, 50000, dict(H=8, Hkv=2, D=128, Dv=128)), (600, 9000, dict(H=32, Hkv=16, D=128, Dv=128)),
                                         (30, 50000, dict(H=4, Hkv=1)), (1400, 9000, dict(H=112, Hkv=2, D=128, Dv=128)),
                                         (4100, 9000, dict(H=20, Hkv=20, D=64, Dv=96))])
@pytest.mark.parametrize("sink", [0, 4000])
def test_prompts_behind_a_sink(n, length, kw, sink, dtype):
    import mla_sparse_top_gb300 as mla
    m = prompt.make([n], kv_lens=[length], scale=1.0, dtype=dtype, **kw)
    z, v = fill(m, 0, length, sink)
    out, lse = prompt.run(m)
    assert mla.heads_device_status(clear=True) == 0
    check(out[:n], lse[:n], z, v, f"sink at {sink}")
