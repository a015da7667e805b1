"""The bounded device waits of the tree attention kernel.  The bound is cut to
1 us, below the first load's latency, so a wait runs out on purpose (nothing on
the GPU is made to fail, the work is only slower than the bound): the status
must show it, and after the bound is restored the next call must repeat, bit
for bit, a call made before."""
import pytest
import torch

from test_gpu_tree import launch, make, upload

pytestmark = pytest.mark.gpu


# many long sequences: all SMs load from HBM at once, and the first waits last several microseconds
@pytest.mark.parametrize("case", [
    dict(act=[3000, 1700] * 24, S1=2, n_q=128),             # cut between teams, merged
    dict(act=[3000, 1700] * 24, S1=1, n_q=128, int8=True),  # codes converted by the attention kernel
])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_identical(case):
    import mla_sparse_top_gb300 as mla
    m = make(30, **case)
    d = upload(m)
    want, out = torch.zeros_like(d["q_nope"]), torch.zeros_like(d["q_nope"])
    ws = launch(m, d, want, None)
    assert mla.tree_device_status(clear=True) == 0
    torch.empty(64 << 20, dtype=torch.float32, device="cuda").fill_(1.0)  # larger than L2: loads come from HBM
    torch.cuda.synchronize()
    mla.set_wait_limit_ns(1000)
    try:
        launch(m, d, out, None, ws)
        status = mla.tree_device_status(clear=True)
    finally:
        mla.set_wait_limit_ns(mla.DEFAULT_WAIT_LIMIT_NS)
    assert status & mla.MLA_DEVICE_TIMEOUT, f"status {status:#x}: no wait ran out under a 1 us bound"
    launch(m, d, out, None, ws)
    assert mla.tree_device_status(clear=True) == 0
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
