"""Waits that run out in prompts of many sequences, whose plan every SM reads from the workspace: the bound is cut to
1 us, far below what the call waits for (nothing on the GPU is made to fail, the work is only slower than the bound).
The status shows it, nothing around the outputs is written, and the next call repeats, bit for bit, one made before."""
import pytest
import torch

from heads_util import check_gpu
import test_gpu_heads_prompt as prompt

pytestmark = pytest.mark.gpu


# one chunk of many whose items are cut: the parts that were not written may not be joined, nor taken for whole items
@pytest.mark.parametrize("before,behind", [(39, 0), (0, 39), (150, 150)])
def test_cut_items_of_many_sequences(before, behind):
    import mla_sparse_top_gb300 as mla
    lens = [3] * before + [200] + [3] * behind
    m = prompt.make(lens, ctx=[10] * before + [60000] + [10] * behind, paged=True, H=16, Hkv=2, D=128, Dv=128, spare=0)
    T = m["q"].shape[0]
    dims = mla.prompt_dims(m["q"], m["k"], m["v"], m["cu_q"], block_table=m["table"])
    ws = torch.empty(mla.mla_prompt_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    outs = torch.full((T + 2048, 16, 128), 5.0, dtype=m["dtype"], device="cuda")
    lses = torch.full((T + 2048, 16), 5.0, device="cuda")
    out, lse = outs[1024:1024 + T], lses[1024:1024 + T]

    def run():
        mla.mla_prompt_attn_fwd(m["q"], m["k"], m["v"], m["cu_q"], out, lse, ws, block_table=m["table"], act_seqs=m["act"],
                                softmax_scale=m["scale"], dims=dims)
        status = mla.heads_device_status(clear=True)
        for t in (outs, lses):
            assert (t[:1024] == 5).all() and (t[1024 + T:] == 5).all()
        return status
    assert run() == 0
    want = out.clone(), lse.clone()
    for _ in range(3):
        mla.set_wait_limit_ns(1000)
        try:
            status = run()
        finally:
            mla.set_wait_limit_ns(mla.DEFAULT_WAIT_LIMIT_NS)
        assert status == mla.MLA_DEVICE_TIMEOUT, f"status {status:#x}: no wait ran out under a 1 us bound"
        assert run() == 0
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for b in {0, before, len(lens) - 1}:
        rows = slice(sum(lens[:b]), sum(lens[:b + 1]))
        k, v = prompt.keys_of(m, b)
        check_gpu(out[rows], lse[rows], m["q"][rows], k.cuda(), v.cuda(), m["scale"], True, f"sequence {b}")
