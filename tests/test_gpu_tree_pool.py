"""Tree attention over a pool much larger than the lengths, its pages spread
over all of it.  From 32,769 blocks on, INT8 rows are not expanded first but
turned into bf16 by the attention kernel, also for three and more row blocks,
several passes and teams; bf16 rows go the same way in any pool."""
import pytest
import torch

from test_gpu_tree import check, launch, make, upload

pytestmark = pytest.mark.gpu
BLOCKS = 40_000


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("act,S1,n_q,lens", [
    ([700, 3, 1500], 3, 128, None),          # three row blocks
    ([900, 40, 0, 2600], 17, 128, [17, 9, 0, 1]),  # one to seventeen, with padding
    ([6000], 40, 128, None),                 # one sequence through all clusters
    ([300] * 40, 5, 100, None),              # many cut row blocks
])
def test_pages_spread_over_a_large_pool(act, S1, n_q, lens, int8):
    import mla_sparse_top_gb300 as mla
    m = make(50 + len(act), act, S1, n_q, int8=int8, lens=lens)
    d = upload(m)
    used = m["kv_nope"].shape[0] // 128
    spread = 1 + torch.randperm(BLOCKS - 2, generator=torch.Generator().manual_seed(3))[:used - 2]
    ids = torch.cat([torch.tensor([0]), spread, torch.tensor([BLOCKS - 1])])  # both ends of the pool among them
    rows = (ids.cuda()[:, None] * 128 + torch.arange(128, device="cuda")).flatten()
    for k, poison in (("kv_nope", 77 if int8 else float("inf")), ("kv_rope", float("nan")), ("kv_scales", float("nan"))):
        if d[k] is not None:
            pool = torch.full((BLOCKS * 128, d[k].shape[1]), poison, dtype=d[k].dtype, device="cuda")
            pool[rows] = d[k]
            d[k] = pool
    table = torch.from_numpy(m["table"])
    d["block_table"] = torch.where(table >= 0, ids[table.clamp(min=0).long()], -1).to(torch.int32).cuda()
    dims = mla.tree_dims(d["q_nope"], d["kv_nope"], d["block_table"], S1=S1)
    assert mla.mla_tree_workspace_bytes(dims) < 64 << 20  # nothing is expanded
    out, again = torch.empty_like(d["q_nope"]), torch.empty_like(d["q_nope"])
    lse = torch.empty(out.shape[:2], device="cuda")
    ws = launch(m, d, out, lse)
    launch(m, d, again, None, ws)
    status = mla.tree_device_status(clear=True)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert check(m, (out.double().cpu().numpy(), lse.double().cpu().numpy(), status)) == 0


def test_binding_refuses_a_transposed_table():
    m = make(60, [100, 300], 1, 16)  # two sequences, tables of three pages
    d = upload(m)
    assert d["block_table"].shape == (2, 3)
    out, lse = torch.empty_like(d["q_nope"]), torch.empty(d["q_nope"].shape[:2], device="cuda")
    for table in (d["block_table"].t(), d["block_table"].t().contiguous().t(), d["block_table"][:, :2]):
        with pytest.raises(ValueError):
            launch(m, {**d, "block_table": table}, out, lse)
