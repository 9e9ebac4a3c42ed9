"""kvc_i4_tree_attn over tiles of 128 query rows where the few rows of a chain would go another way: many units, offsets past
32 bits, groups of zeros, counts outside the capacity."""
import pytest
import torch

import budgeted_kv_cache_gb300 as kvc
from test_gpu_tree_attn import Problem, gen, i32, randn

pytestmark = pytest.mark.gpu
G32, ROW = 0, 1


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()


@pytest.mark.parametrize("n", [33, 150])
def test_many_units(n):
    """65,600 units, one row tile and two; some of them looked at."""
    p = Problem(B=16400, L=1, G=1, H=4, d=64, n=n, counts=(6,) * 16400, spare=0)
    p.call()
    torch.cuda.synchronize()
    small = Problem(B=1, G=1, H=4, d=64, n=n, counts=(6,), spare=0)
    for b in [0, 1, 8191, 16383, 16384, 16399]:
        for name in ("k", "v", "k_scale", "v_scale", "pos", "count", "next_pos"):
            getattr(small.rows, name).copy_(getattr(p.rows, name)[b * 4:b * 4 + 4])
        small.q, small.k, small.v = p.q[b:b + 1].clone(), p.k[b:b + 1].clone(), p.v[b:b + 1].clone()
        small.out, small.lse, small.parents = p.out[b:b + 1], p.lse[b:b + 1], [p.parents[b]]
        small.check()


@pytest.mark.parametrize("n,window", [(20, 0), (20, 300), (150, 0)])
def test_rows_past_32_bit_offsets(n, window):
    """A cache of 40 units of 900,000 rows: 2.3e9 bytes of codes each for keys and values in front of the last unit's."""
    units, cap, d = 40, 900_000, 128
    shape = kvc.make_shape(1, units, 1, 1, d, 1)
    rows = kvc.I4Rows.allocate(shape, cap, mass=False)
    for t in (rows.k, rows.v, rows.k_scale, rows.v_scale, rows.pos):
        t.zero_()
    p = Problem(B=1, L=1, G=1, H=1, d=d, n=n, counts=(500,), spare=0)
    for name in ("k", "v", "k_scale", "v_scale", "pos"):
        getattr(rows, name)[units - 1, :500] = getattr(p.rows, name)[0, :500]
    rows.count[units - 1] = 500
    rows.next_pos[units - 1] = p.rows.next_pos[0]
    q, k, v = (randn(gen(1), 1, units, 1, n, d) for _ in range(3))
    q[0, units - 1], k[0, units - 1], v[0, units - 1] = p.q[0, 0], p.k[0, 0], p.v[0, 0]
    out, lse = torch.zeros_like(q), torch.zeros(1, units, 1, n, device="cuda")
    ws = torch.empty(max(256, kvc.kvc_i4_tree_attn_workspace_bytes(shape, rows, n)), dtype=torch.uint8, device="cuda")
    mods = kvc.ScoreMods(window=window)
    kvc.kvc_i4_tree_attn(shape, rows, q, k, v, p.parent, out, row_lse=lse, mods=mods, workspace=ws)
    p.call(mods=mods)
    torch.cuda.synchronize()
    p.out.copy_(out[:, units - 1:])
    p.lse.copy_(lse[:, units - 1:])
    p.check(window=window)


@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
def test_rows_at_the_end_of_a_long_unit(mode):
    """One unit of 5,000,000 rows: positions of tiles and of scales past 2^22 rows."""
    count = 5_000_000
    p = Problem(B=1, L=1, G=1, H=1, d=64, n=40, counts=(count,), spare=0, mode=mode)
    p.call(mods=kvc.ScoreMods(window=1000)).check(window=1000)


@pytest.mark.parametrize("n", [5, 40])
def test_groups_of_zeros_beside_small_values(n):
    """A group of zeros is stored with a scale of one; it tells nothing about the sizes of the others."""
    p = Problem(B=1, G=4, H=1, n=n, counts=(0,), spare=260)
    g, x = gen(3), []
    for size in (2.0 ** -40, 2.0 ** -45):
        t = randn(g, 1, 1, 1, 260, 128) * size
        t[:, :, :, ::3, :32] = 0
        t[:, :, :, 5] = 0
        t[:, :, :, 64:96] = 0                                  # a quarter of a tile, and a whole one
        t[:, :, :, 128:256] = 0
        x.append(t)
    kvc.kvc_i4_append(p.shape, p.rows, *x)
    p.q *= 2.0 ** 38
    p.k *= 2.0 ** -40
    p.v *= 2.0 ** -45
    p.call().check()


@pytest.mark.parametrize("G,n", [(2, 9), (2, 70)])
def test_counts_outside_the_capacity_are_limited(G, n):
    p = Problem(B=1, G=G, H=2, n=n, counts=(40,), spare=0)
    p.rows.count.copy_(i32([1000, -3]))
    p.call()
    p.rows.count.copy_(i32([40, 0]))
    p.check()


@pytest.mark.parametrize("n", [9, 60, 4])
def test_results_repeat_bit_for_bit(n):
    """Zeros, sizes far apart and splits among them: no result hangs on which warp or block is faster."""
    p = Problem(B=2, G=4, H=2, n=n, counts=(0, 0), spare=4000)
    g = gen(7)
    k, v = (randn(g, 2, 1, 2, 4000, 128) for _ in range(2))
    v[:, :, :, 200:900] = 0
    v[:, :, :, 1500:1700] *= 2.0 ** 60
    kvc.kvc_i4_append(p.shape, p.rows, k, v)
    p.call().check()
    want, lse = p.out.clone(), p.lse.clone()
    for _ in range(20):
        p.call()
        assert torch.equal(p.out, want) and torch.equal(p.lse, lse)
