"""The bounded waits of kvc_prompt_attn: a test hook makes one unit's blocks wait for 16 bytes more than their first key
tile brings.  After the bound that unit reports KVC_UNIT_TIMEOUT, the others' rows are right, and the same call
without the hook succeeds.  Nothing faults: every wait ends, the copies land and tensor memory is freed."""
import pytest
import torch

from test_gpu_prompt_attn import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()
    import budgeted_kv_cache_gb300 as lib
    lib.library()
    return lib


FORMS = {
    "one_tile_of_rows": dict(n_q=30, T=300),
    "two_tiles_of_rows": dict(B=20, Hkv=4, n_q=100, T=700),     # 256 rows of 400 a block
    "documents": dict(n_q=200, T=200, docs=[0] * 90 + [1] * 110),
    "plain_query_loads": dict(n_q=40, T=300, G=3, d=64),
    "split_keys": dict(n_q=1, T=9000),
    "one_key_tile": dict(n_q=1, T=100),
}


@pytest.mark.parametrize("form", FORMS)
def test_a_wait_that_cannot_complete_reports_timeout(kvc, form):
    c = Case(kvc, **FORMS[form])
    c.run()
    torch.cuda.synchronize()
    want, want_lse = c.out.clone(), c.lse.clone()
    c.out.fill_(7.0)
    kvc.kvc_set_overrides(score_stall_unit=1)
    try:
        c.run()
        torch.cuda.synchronize()
    finally:
        kvc.kvc_set_overrides(reset=True)
    status = c.status.tolist()
    assert status[1] == kvc.UNIT_TIMEOUT and sum(status) == kvc.UNIT_TIMEOUT
    heads = [h for h in range(c.Hkv * c.G) if h // c.G != 1]
    for b in range(c.B):
        mine = heads if b == 0 else list(range(c.Hkv * c.G))
        assert torch.equal(c.out[b, 0, mine], want[b, 0, mine]) and torch.equal(c.lse[b, 0, mine], want_lse[b, 0, mine])
    c.status.zero_()
    c.run()
    c.check()
    assert torch.equal(c.out, want)
