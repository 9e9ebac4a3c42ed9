"""kvc_i4_tree_attn where a unit's values come late (a test hook, 20 us a tile): the softmax has long written the weights of
both halves of its last tile when their products begin, so its outputs have to wait for both.  Same results, bit for bit."""
import pytest
import torch

import budgeted_kv_cache_gb300 as kvc
from test_gpu_tree_attn import Problem

pytestmark = pytest.mark.gpu

FORMS = {                                          # cached rows: none to several tiles of 128 for each block
    "one_row_tile": dict(G=4, H=2, n=9),
    "two_row_tiles": dict(G=4, H=2, n=60),
    "row_scales": dict(G=4, H=2, n=9, mode=1),
    "two_row_tiles_row_scales_d_64": dict(G=4, H=2, n=60, d=64, mode=1),
}


@pytest.mark.parametrize("counts", [(0,), (100,), (300,), (2000,), (150,) * 90], ids=lambda c: f"{len(c)}x{c[0]}")
@pytest.mark.parametrize("form", FORMS)
def test_outputs_wait_for_every_product(form, counts):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    p = Problem(B=len(counts), counts=counts, **FORMS[form])
    p.call().check()
    want, want_lse = p.out.clone(), p.lse.clone()
    for unit in (0, 1):
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
        kvc.kvc_set_overrides(select_stall_unit=unit)
        try:
            for _ in range(3):
                p.call()
            torch.cuda.synchronize()
        finally:
            kvc.kvc_set_overrides(reset=True)
        assert torch.equal(p.out, want) and torch.equal(p.lse, want_lse)
        assert p.status.tolist() == [55] * p.status.numel()
