"""The bounded waits of kvc_i4_tree_attn: a test hook makes one unit's blocks wait for key tiles that never come.  After the
bound that unit reports KVC_UNIT_TIMEOUT, the others' rows are right, and the same call without the hook succeeds.  Nothing
faults: every wait ends and tensor memory is freed."""
import pytest
import torch

import budgeted_kv_cache_gb300 as kvc
from test_gpu_tree_attn import Problem

pytestmark = pytest.mark.gpu

FORMS = {
    "one_row_tile_in_splits": dict(B=1, G=4, H=2, n=9, counts=(2000,)),
    "two_row_tiles_in_splits": dict(B=1, G=4, H=2, n=60, counts=(2000,)),
    "one_row_tile": dict(B=20, G=4, H=8, d=64, n=9, counts=(900,) * 20),
    "two_row_tiles": dict(B=20, G=4, H=8, d=64, n=60, counts=(900,) * 20),
    "no_cached_rows": dict(B=1, G=4, H=2, n=9, counts=(0,)),
    "row_scales": dict(B=1, G=4, H=2, n=9, counts=(700,), mode=1),
}


@pytest.mark.parametrize("form", FORMS)
def test_a_wait_that_cannot_complete_reports_timeout(form):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    p = Problem(**FORMS[form]).call()
    torch.cuda.synchronize()
    want, want_lse = p.out.clone(), p.lse.clone()
    p.out.fill_(7.0)
    kvc.kvc_set_overrides(score_stall_unit=1)
    try:
        p.call()
        torch.cuda.synchronize()
    finally:
        kvc.kvc_set_overrides(reset=True)
    status = p.status.tolist()
    assert status[1] == kvc.UNIT_TIMEOUT and status[:1] + status[2:] == [55] * (len(status) - 1)
    for b in range(p.B):
        mine = [h for h in range(p.H * p.G) if b or h // p.G != 1]
        assert torch.equal(p.out[b, 0, mine], want[b, 0, mine]) and torch.equal(p.lse[b, 0, mine], want_lse[b, 0, mine])
    p.status.fill_(55)
    p.call().check()
    assert torch.equal(p.out, want)
