"""kvc_i4_tree_attn over rows whose values differ widely in size: a row whose values are too small to matter for the output
still has its whole share of the row sum, and so of row_lse and of every other row's weight."""
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


def sized(sizes, of_tree, mode=G32, **kw):
    """A problem whose cached values have sizes[j % len] in rows 32 j .. 32 j + 31 (0: zeros), the tree's of_tree."""
    counts = kw.pop("counts")
    p = Problem(counts=(0,) * len(counts), spare=max(counts) + 3, mode=mode, **kw)
    g, n = gen(11), max(counts)
    size = torch.tensor([sizes[j // 32 % len(sizes)] for j in range(n)], device="cuda", dtype=torch.float64)[:, None]
    k, v = (randn(g, p.B, p.L, p.H, n, p.d) for _ in range(2))
    v = (v.double() * size).to(torch.bfloat16)
    kvc.kvc_i4_append(p.shape, p.rows, k, v, n_new=i32(list(counts)))
    p.v.copy_((p.v.double() * of_tree).to(torch.bfloat16))
    return p


BIG, SMALL, TINY = 2.0 ** 90, 2.0 ** -60, 2.0 ** -85
SIZES = {
    "small_behind_big": ((BIG,) * 4 + (SMALL,) * 4, SMALL),
    "big_behind_small": ((SMALL,) * 4 + (BIG,) * 4, SMALL),
    "zeros_behind_big": ((BIG, 0.0), BIG),
    "big_behind_zeros": ((0.0,) * 5 + (BIG,), 1.0),
    "ordinary_then_big": ((1.0,) * 9 + (BIG,), 1.0),
    "ordinary_then_tiny": ((1.0,) * 7 + (TINY,), 1.0),
    "tiny_then_ordinary": ((TINY,) * 7 + (1.0,), TINY),
    "all_kinds": ((TINY, 1.0, 0.0, BIG, SMALL, 2.0 ** 45, 2.0 ** -45), 2.0 ** 30),
    "big_tree": ((SMALL,), BIG),
    "tiny_tree": ((BIG,), TINY),
    "all_tiny": ((TINY,), TINY),
    "all_big": ((BIG,), BIG),
    "all_small": ((SMALL,), SMALL),
    "all_of_2_70": ((2.0 ** 70,), 2.0 ** 66),
    "small_and_zeros": ((SMALL, SMALL, 0.0), SMALL),
    "other_sizes_in_other_splits": ((SMALL,) * 40 + (2.0 ** 70,) * 60, 1.0),
    "at_the_ends": ((2.0 ** 40, 2.0 ** -40, 2.0 ** 55, 2.0 ** -25, 0.0), 2.0 ** 44),
}


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("G,n,d,counts", [(4, 9, 128, (512,)), (4, 60, 128, (512,)), (2, 40, 64, (3000, 700)),
                                          (1, 9, 128, (512,))], ids=["one_row_tile", "two_row_tiles", "splits", "few_rows"])
def test_sums_of_rows_of_any_size(sizes, G, n, d, counts):
    sizes, tree = SIZES[sizes]
    sized(sizes, tree, B=len(counts), G=G, H=2, n=n, d=d, counts=counts).call().check()


@pytest.mark.parametrize("sizes", ["small_behind_big", "big_behind_zeros", "all_kinds"])
@pytest.mark.parametrize("n", [9, 60])
def test_without_splits(sizes, n):
    sizes, tree = SIZES[sizes]
    sized(sizes, tree, B=20, G=4, H=8, n=n, d=64, counts=(400,) * 10 + (257,) * 10).call().check()


@pytest.mark.parametrize("tree", [BIG, TINY])
@pytest.mark.parametrize("n", [9, 60])
def test_row_scales(tree, n):
    """Cached values of fp16's range beside a tree's of bf16's."""
    sized((2.0 ** 12, 2.0 ** -12, 0.0), tree, mode=ROW, G=4, H=2, n=n, counts=(700,)).call().check()


@pytest.mark.parametrize("n", [9, 60])
def test_with_modifiers(n):
    sizes, tree = SIZES["all_kinds"]
    slopes = torch.tensor([2.0 ** -(h + 3) for h in range(8)], device="cuda")
    p = sized(sizes, tree, G=4, H=2, n=n, counts=(1500,))
    p.call(mods=kvc.ScoreMods(20.0, slopes, 900, i32([70]))).check(softcap=20.0, slopes=slopes, window=900, prefix=[70])


def test_many_tiny_rows():
    """600,000 equal weights of values whose exponent is near the least: the sum is finite and counts them all."""
    for size in (2.0 ** -88, 2.0 ** -70):
        p = sized((size,), size, G=1, H=1, n=20, d=64, counts=(600_000,))
        p.q.zero_()
        p.call().check()
