"""A head whose norm is not finite stays alone: every other head has the bits that it has without it."""
import pytest
import torch

from heads_util import TYPES
from test_gpu_heads_prep import inputs, make_norm

pytestmark = pytest.mark.gpu


def spoil(x, off, rot):
    """NaN, infinities and zeros in heads that others of their token follow; returns the heads."""
    T, H, D = x.shape
    plain = next((d for d in range(D) if not off <= d < off + rot), 0)  # a value that does not turn, where there is one
    heads = []
    for t, h, d, value in ((0, 0, 0, float("nan")), (T // 3, 1 % H, plain, float("inf")), (T // 2, 0, D - 1, -float("inf")),
                           (T - 1, H // 2, plain, float("nan"))):
        x[t, h, d] = value
        heads.append((t, h))
    x[T // 4, 2 % H] = 0
    return heads + [(T // 4, 2 % H)]


# heads of single values in one pass of a group and in several, and heads of 16-byte units; tokens and
# heads enough for a group to take nine and more heads of a token, one after the other
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind,eps", [("rms", 0.0), ("rms", 1e-6), ("layer", 0.0)])
@pytest.mark.parametrize("T,H,D,off,rot,pad", [(1300, 17, 107, 7, 36, 5), (2600, 18, 33, 0, 16, 3), (1300, 17, 61, 0, 0, 0),
                                               (900, 20, 128, 32, 64, 1), (900, 20, 128, 32, 64, 0), (300, 12, 1111, 3, 30, 1)])
def test_heads_stay_alone(T, H, D, off, rot, pad, kind, eps, dtype):
    import mla_sparse_top_gb300 as mla
    x, pos = inputs(T, H, D, TYPES[dtype], pad, seed=T + D)
    own = make_norm(kind, D, x.dtype, fp32=False, seed=D, eps=eps)[1]
    for half in (False, True):
        def run():
            y = torch.empty((T, H, D), dtype=x.dtype, device="cuda")
            mla.mla_norm_rope(pos, x, params=mla.rope_params(), out=y, q_norm=own, rot_dim=rot, rot_off=off, half=half)
            return y
        before = x.clone()
        clean = run()
        bad = spoil(x, off, rot)
        got = run()
        x.copy_(before)
        same = torch.ones((T, H), dtype=torch.bool, device="cuda")
        for t, h in bad:
            same[t, h] = False
            if eps == 0 or (t, h) != bad[-1]:
                assert not torch.isfinite(got[t, h]).all(), (t, h)
        wrong = (same & (got != clean).any(-1)).nonzero()
        assert wrong.numel() == 0, f"half {half}: heads {wrong[:5].tolist()} changed"
    assert mla.heads_device_status(clear=True) == 0


def test_appended_keys_stay_alone():
    """The same of queries, keys and values that one call writes, LayerNorm beside the RMS norm."""
    import mla_sparse_top_gb300 as mla
    T, H, Hkv, D, rot = 1300, 21, 12, 75, 20
    q, pos = inputs(T, H, D, torch.bfloat16, 2, seed=1)
    k, _ = inputs(T, Hkv, D, torch.bfloat16, 2, seed=2)
    v, _ = inputs(T, Hkv, D, torch.bfloat16, 2, seed=3)
    rows = torch.arange(T).cuda()

    def run(q_kind):
        kc, vc = (torch.zeros((11, 128, Hkv, D), dtype=q.dtype, device="cuda") for _ in range(2))
        out = torch.empty((T, H, D), dtype=q.dtype, device="cuda")
        mla.mla_kv_append(pos, rows, k, v, kc, vc, params=mla.rope_params(), rot_dim=rot, rot_off=3, half=True, q=q, q_out=out,
                          k_norm=make_norm("rms", D, q.dtype, True, eps=0.0)[1], q_norm=make_norm(q_kind, D, q.dtype, True, eps=0.0)[1])
        return out, kc.flatten(0, 1)[:T], vc.flatten(0, 1)[:T]
    for q_kind in ("rms", "layer"):
        before = q.clone(), k.clone()
        clean = run(q_kind)
        bad = spoil(q, 3, rot), spoil(k, 3, rot)
        got = run(q_kind)
        q.copy_(before[0]), k.copy_(before[1])
        assert torch.equal(got[2], clean[2])
        for i, heads in enumerate(bad):
            same = torch.ones(got[i].shape[:2], dtype=torch.bool, device="cuda")
            for t, h in heads:
                same[t, h] = False
            assert torch.equal(got[i][same], clean[i][same]), (q_kind, i)
    assert mla.heads_device_status(clear=True) == 0
