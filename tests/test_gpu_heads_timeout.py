"""Waits that run out in calls on ordinary heads: the bound is cut to 1 us, far below what the calls wait for (nothing
on the GPU is made to fail, the work is only slower than the bound).  The status shows it, nothing outside the outputs
is written, and the next call repeats, bit for bit, one made before."""
import pytest
import torch

import test_gpu_heads_paged as paged
import test_gpu_heads_prompt as prompt

pytestmark = pytest.mark.gpu


def short_then_whole(run, want):
    import mla_sparse_top_gb300 as mla
    assert mla.heads_device_status(clear=True) == 0
    torch.empty(64 << 20, dtype=torch.float32, device="cuda").fill_(1.0)  # larger than L2: loads come from HBM
    torch.cuda.synchronize()
    mla.set_wait_limit_ns(1000)
    try:
        run()
        status = mla.heads_device_status(clear=True)
    finally:
        mla.set_wait_limit_ns(mla.DEFAULT_WAIT_LIMIT_NS)
    assert status == mla.MLA_DEVICE_TIMEOUT, f"status {status:#x}: no wait ran out under a 1 us bound"
    got = run()
    assert mla.heads_device_status(clear=True) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# all SMs load from HBM at once, and the first waits last several microseconds: heads cut and joined, by every
# warp's own plan and by the block's
@pytest.mark.parametrize("act,kw", [([9000, 5000] * 12, dict(H=32, Hkv=8)), ([6000, 70, 3000] * 16, dict(H=32, Hkv=8)),
                                    ([9000, 5000] * 12, dict(S1=5, H=40, Hkv=8, D=96, Dv=96))])
def test_new_tokens(act, kw):
    m = paged.make(act, **kw)
    short_then_whole(lambda: paged.run(m), paged.run(m))
