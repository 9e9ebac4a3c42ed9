"""kvc_rope_tables at the last positions that there are (GPU): 2^31 - 1 rows of 8 pairs, 137 GB of tables."""
from decimal import Decimal, getcontext

import pytest
import torch

import budgeted_kv_cache_gb300 as kvc

pytestmark = pytest.mark.gpu


def test_the_last_positions():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()
    torch.cuda.empty_cache()
    n, rot, base = 2 ** 31 - 1, 16, 1000000
    if torch.cuda.mem_get_info()[0] < 150 * 2 ** 30:
        pytest.skip("no room for the tables")
    cos, sin = torch.empty(n, rot // 2, device="cuda"), torch.empty(n, rot // 2, device="cuda")
    kvc.kvc_rope_tables(cos, sin, float(base))
    at = list(range(n - 300, n)) + [2 ** 30 - 1, 2 ** 30, 2 ** 29 + 12345, 2 ** 31 - 2 ** 20] + list(range(5))
    getcontext().prec = 50
    tau = 2 * Decimal("3.14159265358979323846264338327950288419716939937510")
    theta = [Decimal(base) ** (Decimal(-2 * i) / rot) for i in range(rot // 2)]
    x = torch.tensor([[float(p * t % tau) for t in theta] for p in at], dtype=torch.float64)
    rows = torch.tensor(at, device="cuda")
    got = cos[rows].double().cpu(), sin[rows].double().cpu()
    del cos, sin
    torch.cuda.empty_cache()
    # the documented bound (the reference's own angle is off by 2^-51)
    for have, want in zip(got, (x.cos(), x.sin())):
        assert float((have - want).abs().max()) <= 2.0 ** -22
