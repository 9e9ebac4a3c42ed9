"""kvc_i4_tree_attn against 64-bit attention over the cached rows and each node's ancestors (GPU)."""
import math

import pytest
import torch

import budgeted_kv_cache_gb300 as kvc
from attn_reference import close
from tree_reference import tree_attention, trees

pytestmark = pytest.mark.gpu
G32, ROW = 0, 1


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def randn(g, *s):
    return torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)


class Problem:
    """Rows, a tree's tensors and the call; counts [B] rows in use."""

    def __init__(self, B=1, L=1, G=4, H=2, d=128, n=5, counts=(100,), mode=G32, kind="random", seed=0, by_token=False, spare=3,
                 k_size=1.0, v_size=1.0):
        self.B, self.L, self.G, self.H, self.d, self.n, self.seed = B, L, G, H, d, n, seed
        g = self.g = gen(seed)
        cap = max(counts) + spare
        self.shape = kvc.make_shape(B, L, G * H, H, d, 1)
        self.rows = kvc.I4Rows.allocate(self.shape, cap, mode)
        for t in (self.rows.k, self.rows.v):
            t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
        for t in (self.rows.k_scale, self.rows.v_scale, self.rows.mass):
            t.fill_(float("nan"))
        self.rows.pos.fill_(-7)
        if max(counts):
            x = [randn(g, B, L, H, max(counts), d) * s for s in (k_size, v_size)]
            kvc.kvc_i4_append(self.shape, self.rows, *x, n_new=i32(list(counts)))
        gap = torch.randint(1, 4, self.rows.pos.shape, generator=g, device="cuda")
        pos = (torch.cumsum(gap, 1) - gap).to(torch.int32)
        used = torch.arange(cap, device="cuda") < self.rows.count[:, None]
        self.rows.pos.copy_(torch.where(used, pos, self.rows.pos))
        self.rows.next_pos.copy_(torch.where(used, pos + 1, 0).amax(1))
        shape = lambda heads: (B, L, n, heads, d) if by_token else (B, L, heads, n, d)
        turn = (lambda t: t.transpose(2, 3)) if by_token else (lambda t: t)
        self.q = turn(randn(g, *shape(G * H)) * 2.0)
        self.k, self.v = turn(randn(g, *shape(H)) * k_size), turn(randn(g, *shape(H)) * v_size)
        self.parents = [trees(kind, n, seed + b) for b in range(B)]
        self.parent = i32(self.parents)
        self.out = turn(torch.full(shape(G * H), 7.0, dtype=torch.bfloat16, device="cuda"))
        self.lse = torch.full((B, L, G * H, n), 7.0, device="cuda")
        self.status = torch.full((B * L * H,), 55, dtype=torch.int32, device="cuda")
        self.space()

    def space(self):
        self.ws = torch.full((max(256, kvc.kvc_i4_tree_attn_workspace_bytes(self.shape, self.rows, self.n)),), 255,
                             dtype=torch.uint8, device="cuda")

    def call(self, **kw):
        kvc.kvc_i4_tree_attn(self.shape, self.rows, self.q, self.k, self.v, self.parent, self.out, row_lse=self.lse,
                             unit_status=self.status, workspace=self.ws, **kw)
        return self

    def check(self, sizes=None, scale=None, status=55, **mods):
        torch.cuda.synchronize()
        G = self.G
        slopes, prefix = mods.pop("slopes", None), mods.pop("prefix", [-2 ** 40] * self.B)
        for b in range(self.B):
            m = self.n if sizes is None else max(0, min(self.n, sizes[b]))
            for l in range(self.L):
                for h in range(self.H):
                    u = (b * self.L + l) * self.H + h
                    here = slice(h * G, h * G + G)
                    out, lse = self.out[b, l, here], self.lse[b, l, here]
                    assert bool((out[:, m:] == 7).all()) and bool((lse[:, m:] == 7).all())
                    if m == 0:
                        continue
                    want = tree_attention(self.rows, u, self.q[b, l, here, :m].double(), self.k[b, l, h, :m].double(),
                                          self.v[b, l, h, :m].double(), self.parents[b][:m], scale or 1 / math.sqrt(self.d),
                                          slopes=None if slopes is None else slopes[here], prefix=prefix[b], **mods)
                    close(out[:, :m], want[0], want[3], f"out of unit {u}")
                    close(lse[:, :m], want[1], want[4], f"lse of unit {u}")
        assert self.status.tolist() == [status] * self.status.numel()


@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,kind", [(1, "roots"), (2, "chain"), (13, "random"), (64, "random"), (40, "star"), (130, "random")])
def test_trees(n, kind, d, mode):
    Problem(B=2, G=4, H=2, d=d, n=n, counts=(300, 129), mode=mode, kind=kind, seed=n).call().check()


@pytest.mark.parametrize("counts", [(0,), (1,), (127,), (128,), (129,), (255, 0, 1), (2304, 2000), (9001, 3)], ids=str)
@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
def test_lengths(counts, mode):
    Problem(B=len(counts), G=4, H=1, n=7, counts=counts, mode=mode).call().check()


@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
@pytest.mark.parametrize("n,window", [(9, 0), (40, 0), (40, 500), (9, 500), (4, 0), (2, 500), (8, 500)])
def test_units_that_fill_the_gpu(n, window, mode):
    """Every block walks many tiles: one row tile's two streams take them in turn, two row tiles share them."""
    p = Problem(B=20, G=4, H=8, d=64, n=n, counts=[1500 - 61 * b for b in range(20)], mode=mode, seed=9)
    p.call(mods=kvc.ScoreMods(window=window)).check(window=window)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 33])
@pytest.mark.parametrize("n", [1, 9, 51])
def test_groups(G, n):
    Problem(B=1, L=2, G=G, H=3, d=64, n=n, counts=(200,), seed=G).call().check()


def test_blocks_in_the_order_of_their_lengths():
    """More blocks than SMs, several row tiles a unit, equal and empty units among them."""
    Problem(B=13, G=4, H=4, d=64, n=150, counts=[700 * (b % 5) for b in range(13)], seed=5).call().check()


@pytest.mark.parametrize("n,kind", [(256, "random"), (300, "chain"), (1024, "random"), (1024, "chain")])
def test_large_trees(n, kind):
    Problem(G=2, H=1, n=n, counts=(700,), kind=kind, d=64).call().check()


def test_strides():
    Problem(B=3, L=2, G=3, H=2, n=21, counts=(140, 5, 333), by_token=True).call().check()


@pytest.mark.parametrize("G,n,d", [(4, 33, 128), (1, 16, 128), (2, 16, 64), (4, 4, 64)])
def test_padded_trees(G, n, d):
    p = Problem(B=5, G=G, H=2, n=n, d=d, counts=(150, 20, 129, 0, 7))
    sizes = [n, 0, 1, n // 2, 999]
    for b, m in enumerate(sizes):                              # what is no node may hold any bits
        p.q[b, :, :, m:] = float("nan")
        p.k[b, :, :, m:] = float("nan")
        p.v[b, :, :, m:] = float("inf")
        p.parent[b, m:] = 12345
    p.call(n_nodes=i32(sizes)).check(sizes)


MODS = [dict(softcap=20.0), dict(softcap=1.0), dict(slopes=True), dict(window=1), dict(window=5), dict(window=130),
        dict(window=60, prefix=True), dict(softcap=30.0, slopes=True, window=500, prefix=True), dict(softcap=5000.0),
        dict(softcap=1e-30)]


@pytest.mark.parametrize("mods", MODS, ids=lambda m: "-".join(f"{k}{v}" for k, v in m.items()))
@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
@pytest.mark.parametrize("G,n,d", [(4, 20, 64), (4, 2, 128), (1, 15, 128), (2, 13, 64)])
def test_modifiers(mods, mode, G, n, d):
    """Over the tiles of 128 query rows, and over few rows."""
    p = Problem(B=2, G=G, H=2, d=d, n=n, counts=(700, 129), mode=mode, kind="random", seed=3)
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(2 * G)], device="cuda") if mods.get("slopes") else None
    prefix = [90, 3] if mods.get("prefix") else None
    m = kvc.ScoreMods(mods.get("softcap", 0.0), slopes, mods.get("window", 0), None if prefix is None else i32(prefix))
    p.call(mods=m).check(softcap=mods.get("softcap", 0.0), slopes=slopes, window=mods.get("window", 0), prefix=prefix or [0, 0])


def test_long_window_in_a_long_cache():
    p = Problem(B=2, G=4, H=1, n=30, counts=(9000, 5000), seed=8)
    p.call(mods=kvc.ScoreMods(window=777)).check(window=777)


def test_rows_in_any_order():
    """Eviction leaves rows in any order of their positions: a window looks at the positions, not at the slots."""
    p = Problem(B=1, G=2, H=2, n=11, counts=(1000,), seed=4)
    for u in range(2):
        order = torch.randperm(1000, generator=gen(u), device="cuda")
        for t in (p.rows.k, p.rows.v, p.rows.k_scale, p.rows.v_scale, p.rows.pos):
            t[u, :1000] = t[u, :1000][order]
    p.call(mods=kvc.ScoreMods(window=300)).check(window=300)


def test_blocks_in_the_order_of_their_lengths():
    """More blocks than SMs, several row tiles a unit, equal and empty units among them."""
    counts = [700 * (b % 5) for b in range(13)]
    p = Problem(B=13, G=4, H=4, d=64, n=150, counts=counts, seed=5)
    p.call().check()


@pytest.mark.parametrize("G,n", [(1, 9), (4, 20)])
@pytest.mark.parametrize("nxt", [2 ** 31 - 30, 0, -2 ** 31 + 2000])
def test_positions_over_all_of_int32(G, n, nxt):
    """Distances past 31 bits: far rows are outside a window, and slopes of 2^-30 still tell them apart."""
    p = Problem(B=1, G=G, H=2, n=n, counts=(700,), seed=6)
    pos = torch.randint(-2 ** 31, nxt, (2, 700), generator=gen(3), device="cuda")
    pos[:, :300] = nxt - 1 - torch.arange(300, device="cuda")
    pos[:, 300] = -2 ** 31
    p.rows.pos[:, :700] = pos.to(torch.int32)
    p.rows.next_pos.fill_(nxt)
    p.call(mods=kvc.ScoreMods(window=250)).check(window=250)
    slopes = torch.full((2 * G,), 2.0 ** -30, device="cuda")
    p.call(mods=kvc.ScoreMods(slopes=slopes)).check(slopes=slopes)
    slopes = torch.full((2 * G,), 0.5, device="cuda")
    p.call(mods=kvc.ScoreMods(slopes=slopes, window=2 ** 31 - 1)).check(slopes=slopes, window=2 ** 31 - 1)


def test_scale_and_missing_outputs():
    p = Problem(n=6)
    kvc.kvc_i4_tree_attn(p.shape, p.rows, p.q, p.k, p.v, p.parent, p.out, softmax_scale=0.3, workspace=p.ws)
    p.lse.copy_(p.lse)
    want = p.out.clone()
    p.call(softmax_scale=0.3).check(scale=0.3)
    assert torch.equal(p.out, want)


@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
@pytest.mark.parametrize("k_size,v_size", [(2.0 ** -20, 2.0 ** -30), (2.0 ** 5, 2.0 ** 40), (2.0 ** -100, 2.0 ** -110), (1.0, 2.0 ** 90)])
def test_sizes_of_values(mode, k_size, v_size):
    """Keys and values far from one (fp16 scales end at 2^-24 and 2^15: there the rows are scaled within)."""
    if mode == ROW:
        k_size, v_size = max(k_size, 2.0 ** -10), min(max(v_size, 2.0 ** -12), 2.0 ** 12)
    Problem(B=1, G=4, H=2, n=9, counts=(400,), mode=mode, k_size=k_size, v_size=v_size, seed=5).call().check()


def test_groups_of_zeros_beside_small_values():
    """A group of zeros is stored with a scale of one; it tells nothing about the sizes of the others."""
    p = Problem(B=1, G=4, H=1, n=4, counts=(0,), spare=260)
    g, x = gen(3), []
    for size in (2.0 ** -40, 2.0 ** -45):
        t = randn(g, 1, 1, 1, 260, 128) * size
        t[:, :, :, ::3, :32] = 0
        t[:, :, :, 5] = 0
        x.append(t)
    kvc.kvc_i4_append(p.shape, p.rows, *x)
    p.q *= 2.0 ** 38
    p.k *= 2.0 ** -40
    p.v *= 2.0 ** -45
    p.call().check()


@pytest.mark.parametrize("G", [1, 2])
def test_parents_that_are_no_earlier_node(G):
    p = Problem(B=3, L=1, G=G, H=2, n=12, counts=(50, 60, 70))
    for i, bad in ((3, 3), (5, 8), (7, -2), (9, 2 ** 31 - 1), (10, -2 ** 31)):
        p.parent[1, i] = bad
        p.parents[1][i] = -1
    p.call()
    torch.cuda.synchronize()
    assert p.status.tolist() == [55, 55, kvc.UNIT_BAD_INDEX, kvc.UNIT_BAD_INDEX, 55, 55]
    p.status.fill_(55)
    p.check()


def test_counts_outside_the_capacity_are_limited():
    p = Problem(B=1, G=2, H=2, n=3, counts=(40,), spare=0)
    p.rows.count.copy_(i32([1000, -3]))
    p.call()
    p.rows.count.copy_(i32([40, 0]))
    p.check()


@pytest.mark.parametrize("G", [4, 1])
def test_capture_streams_and_repeats(G):
    p = Problem(B=2, G=G, H=2, n=17, counts=(3000, 1200))
    p.call()
    torch.cuda.synchronize()
    first, lse = p.out.clone(), p.lse.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    p.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.call()
    side.synchronize()
    assert torch.equal(p.out, first) and torch.equal(p.lse, lse)
    with torch.cuda.graph(graph):
        p.call()
        p.call()
    for step in range(3):                                      # other inputs, counts and trees in the same graph
        p.q.copy_(randn(gen(100 + step), *p.q.shape) * 2)
        p.rows.count.copy_(i32([2000 - step * 999, 1, 128 * (step + 1), 900]))
        p.parents = [trees(["chain", "star", "random"][step], p.n, 7 + b) for b in range(2)]
        p.parent.copy_(i32(p.parents))
        graph.replay()
        p.check()


def test_two_calls_at_once():
    a, b = Problem(B=4, G=4, H=4, n=16, counts=(4000,) * 4, seed=1), Problem(B=4, G=4, H=4, n=16, counts=(4000,) * 4, seed=2)
    sides = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip((a, b), sides):
            with torch.cuda.stream(s):
                p.call()
    a.check()
    b.check()


def test_many_units():
    """More units than a grid's second dimension holds."""
    p = Problem(B=16400, L=1, G=1, H=4, d=64, n=2, counts=(6,) * 16400, spare=0)
    p.call()
    torch.cuda.synchronize()
    at = torch.arange(0, 16400, 37)
    small = Problem(B=1, G=1, H=4, d=64, n=2, counts=(6,), spare=0)
    for b in [0, 16383, 16384, 16399] + at[:20].tolist():
        for name in ("k", "v", "k_scale", "v_scale", "pos", "count", "next_pos"):
            getattr(small.rows, name).copy_(getattr(p.rows, name)[b * 4:b * 4 + 4])
        small.q, small.k, small.v = p.q[b:b + 1].clone(), p.k[b:b + 1].clone(), p.v[b:b + 1].clone()
        small.out, small.lse, small.parents = p.out[b:b + 1], p.lse[b:b + 1], [p.parents[b]]
        small.check()


def test_rows_past_32_bit_offsets():
    """A cache of 40 units of 900,000 rows: 2.3e9 bytes of codes each for keys and values."""
    U, cap, d = 40, 900_000, 128
    shape = kvc.make_shape(1, U, 1, 1, d, 1)
    rows = kvc.I4Rows.allocate(shape, cap, mass=False)
    for t in (rows.k, rows.v, rows.k_scale, rows.v_scale, rows.pos):
        t.zero_()
    g = gen(1)
    p = Problem(B=1, L=1, G=1, H=1, d=d, n=5, counts=(500,), spare=0)
    for name in ("k", "v", "k_scale", "v_scale", "pos"):       # the last unit holds rows; others only zeros (a scale of 0)
        getattr(rows, name)[U - 1, :500] = getattr(p.rows, name)[0, :500]
    rows.count[U - 1] = 500
    rows.next_pos[U - 1] = p.rows.next_pos[0]
    q, k, v = (randn(g, 1, U, 1, 5, d) for _ in range(3))
    q[0, U - 1], k[0, U - 1], v[0, U - 1] = p.q[0, 0], p.k[0, 0], p.v[0, 0]
    out = torch.zeros_like(q)
    ws = torch.empty(max(256, kvc.kvc_i4_tree_attn_workspace_bytes(shape, rows, 5)), dtype=torch.uint8, device="cuda")
    kvc.kvc_i4_tree_attn(shape, rows, q, k, v, p.parent, out, workspace=ws)
    p.call()
    torch.cuda.synchronize()
    p.out.copy_(out[:, U - 1:])
    p.check()
