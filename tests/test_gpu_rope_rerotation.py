"""kvc_rope and the compaction's re-rotation turn a pair by the same fp32 operations (GPU): given the cosines and sines that
the compaction forms from its tables, kvc_rope gives its keys bit for bit.  And kvc_rope's difference along a direction is the
rotation of that direction."""
import pytest
import torch

import budgeted_kv_cache_gb300 as kvc
from test_gpu_rope import angles

pytestmark = pytest.mark.gpu
HALF, PAIRS = kvc.ROPE_SPLIT_HALF, kvc.ROPE_INTERLEAVED


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()


@pytest.mark.parametrize("d,rot,layout", [(128, 128, HALF), (128, 128, PAIRS), (64, 64, HALF), (64, 32, PAIRS), (128, 48, HALF),
                                          (64, 16, PAIRS)])
def test_keys_of_a_compaction(d, rot, layout):
    B, L, H, T, n = 2, 1, 2, 700, 300
    U = B * L * H
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(B, L, H, T, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pos = (torch.cumsum(torch.randint(1, 5, (U, T), generator=g, device="cuda"), 1) - 1).to(torch.int32)
    kept = torch.zeros(3, U, n, dtype=torch.int32, device="cuda")
    kept[2] = torch.stack([torch.randperm(T, generator=g, device="cuda")[:n].sort().values for _ in range(U)]).to(torch.int32)
    count = torch.zeros(3, U, dtype=torch.int32, device="cuda")
    count[2] = n
    cos, sin = torch.empty(4096, rot // 2, device="cuda"), torch.empty(4096, rot // 2, device="cuda")
    kvc.kvc_rope_tables(cos, sin, 10000.0)
    shape = kvc.make_shape(B, L, 2 * H, H, d, T)
    pol = kvc.Policy(budget_tokens=n, capacity=n, renumber=True, rope_layout=layout, rotary_dim=rot)
    pools = kvc.Pools.allocate(shape, pol)
    status = torch.zeros(U, dtype=torch.int32, device="cuda")
    kvc.kvc_compact_rerotate_quant(shape, pol, k, v, pos, kept, count, cos, sin, 4096, pools, status)
    assert int(status.abs().sum()) == 0
    one = kvc.make_shape(1, 1, 1, 1, d, 1)
    new = torch.arange(n, device="cuda")
    for u in range(U):
        rows = kept[2, u].long()
        old = pos[u, rows].long()
        # C = c'c + s's, S = s'c - c's, both over the root of C C + S S, an operation at a time
        C = cos[new] * cos[old] + sin[new] * sin[old]
        S = sin[new] * cos[old] - cos[new] * sin[old]
        size = torch.sqrt(C * C + S * S)
        x = k.view(U, T, d)[u, rows][None, None, None].contiguous()
        kvc.kvc_rope(one, None, x, new.to(torch.int32)[None], (C / size).contiguous(), (S / size).contiguous(), rope_layout=layout,
                     rotary_dim=rot)
        assert torch.equal(x[0, 0, 0], pools.k_bf16[u, :n]), u


@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("inverse", [False, True])
def test_differences_along_a_direction(layout, inverse):
    """(R(x + e) - R(x - e)) / 2 against the 64-bit rotation of e, at a random x; the inputs are exact in bf16."""
    n, d, rot = 50, 64, 48
    g = torch.Generator(device="cuda").manual_seed(5)
    # multiples of 1/16 below 8: sums with directions of +-1/2 have 8 bits
    x = torch.randint(-100, 101, (1, 1, 3, n, d), generator=g, device="cuda").double() / 16
    e = (torch.randint(0, 2, x.shape, generator=g, device="cuda").double() * 2 - 1) / 2
    up, down = (x + e).to(torch.bfloat16), (x - e).to(torch.bfloat16)
    assert torch.equal(up.double(), x + e) and torch.equal(down.double(), x - e)
    cos, sin = torch.empty(2000, rot // 2, device="cuda"), torch.empty(2000, rot // 2, device="cuda")
    kvc.kvc_rope_tables(cos, sin, 10000.0)
    pos = torch.randint(0, 2000, (1, n), generator=g, device="cuda", dtype=torch.int32)
    shape = kvc.make_shape(1, 1, 3, 3, d, 1)
    for t in (up, down):
        kvc.kvc_rope(shape, t, None, pos, cos, sin, rope_layout=layout, rotary_dim=rot, inverse=inverse)
    angle = pos[0].double()[:, None] * angles(rot, 10000.0, kvc.RopeScaling()).cuda()
    c, s = angle.cos(), angle.sin() * (-1 if inverse else 1)
    a, b = (e[..., :rot // 2], e[..., rot // 2:rot]) if layout == HALF else (e[..., 0:rot:2], e[..., 1:rot:2])
    y, z = a * c - b * s, b * c + a * s
    want = torch.cat((y, z) if layout == HALF else (torch.stack((y, z), -1).flatten(-2),), -1)
    want = torch.cat((want, e[..., rot:]), -1)
    got = (up.double() - down.double()) / 2
    # each result is off by 2^-8 of itself and by the tables' 2^-22 and fp32's of its pair (below 2 x 10)
    bound = (2.0 ** -8 * (up.double().abs() + down.double().abs()) + 2 * 20 * 2.0 ** -21) / 2
    assert bool(((got - want).abs() <= bound).all())
