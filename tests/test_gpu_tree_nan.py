"""A query row of NaN or infinities: its outputs and its statistics are NaN, so that nothing takes it for a row that saw
nothing (whose statistics are -inf); the other rows are as they were."""
import pytest
import torch

import budgeted_kv_cache_gb300 as kvc
from test_gpu_tree_attn import Problem
from test_gpu_tree_commit import Commit

pytestmark = pytest.mark.gpu

FORMS = {
    "one_row_tile_in_splits": dict(B=1, G=4, H=2, n=9, counts=(2000,)),
    "two_row_tiles_in_splits": dict(B=1, G=4, H=2, n=60, counts=(2000,)),
    "one_row_tile": dict(B=20, G=4, H=8, d=64, n=9, counts=(900,) * 20),
    "two_row_tiles": dict(B=20, G=4, H=8, d=64, n=60, counts=(900,) * 20),
    "row_scales": dict(B=1, G=4, H=2, n=9, counts=(700,), mode=1),
    "few_rows_in_splits": dict(B=1, G=4, H=2, n=4, counts=(2000,)),
    "few_rows": dict(B=20, G=4, H=8, d=64, n=4, counts=(70,) * 20),
    "few_rows_row_scales": dict(B=1, G=1, H=2, n=9, counts=(70,), mode=1),
}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("form", FORMS)
def test_statistics_of_a_row_of_nan(form, value):
    p = Problem(**FORMS[form]).call()
    torch.cuda.synchronize()
    want, want_lse = p.out.clone(), p.lse.clone()
    p.q[0, 0, 1, 2] = value
    p.call()
    torch.cuda.synchronize()
    assert bool(p.out[0, 0, 1, 2].isnan().all()) and bool(p.lse[0, 0, 1, 2].isnan())
    p.out[0, 0, 1, 2], p.lse[0, 0, 1, 2] = want[0, 0, 1, 2], want_lse[0, 0, 1, 2]
    assert torch.equal(p.out, want) and torch.equal(p.lse, want_lse)


@pytest.mark.parametrize("steps,G", [(3, 4), (9, 4)])
def test_mass_of_a_row_of_nan(steps, G):
    """Its weights are not silently left out."""
    p = Commit(steps=steps, B=1, G=G, H=2, n=12, counts=(150,), spare=steps, kind="chain").commit()
    torch.cuda.synchronize()
    kept = p.rows.mass.clone()
    for t, t0 in zip((p.rows.mass, p.rows.count, p.rows.next_pos), (p.before[5], p.before[6], p.before[7])):
        t.copy_(t0)
    p.q[0, 0, 1, 1] = float("nan")                             # of the first KV head
    p.call()
    p.again()
    torch.cuda.synchronize()
    assert bool(p.rows.mass[0, :152].isnan().all())
    # the others' statistics are the call's own here, and were the 64-bit ones: 1e-5 apart at most, as their weights
    for now, was in ((p.rows.mass[0, 152:150 + steps], kept[0, 152:150 + steps]), (p.rows.mass[1, :150 + steps], kept[1, :150 + steps])):
        assert bool(((now - was).abs() <= 2e-5 * was + 1e-6).all())
