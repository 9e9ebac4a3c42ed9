"""kvc_i4_tree_commit against the oracle's quantiser and 64-bit softmax weights, and trees checked, committed and evicted in
turn (GPU)."""
import math

import numpy as np
import pytest
import torch

import budgeted_kv_cache_gb300 as kvc
import oracle as o
from attn_reference import U, close
from test_gpu_tree_attn import Problem, gen, i32, randn
from tree_reference import held, lines, path_mass, trees

pytestmark = pytest.mark.gpu
G32, ROW = 0, 1


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()


def fields(r):
    return [t for t in (r.k, r.v, r.k_scale, r.v_scale, r.pos, r.mass, r.count, r.next_pos) if t is not None]


def bits(t):
    return t.contiguous().view(torch.uint8)


class Commit(Problem):
    """A problem with an accepted path; the call's outputs are checked against `before`."""

    def __init__(self, steps=4, sizes=None, **kw):
        super().__init__(**kw)
        self.steps = steps
        self.sizes = sizes or [steps] * self.B
        self.paths = []
        for b in range(self.B):
            way = max(lines(self.parents[b]), key=len)[:max(0, min(steps, self.sizes[b]))]
            self.paths.append(way)
        self.sizes = [min(len(w), s) if s >= 0 else s for w, s in zip(self.paths, self.sizes)]
        self.path = i32([w + [10 ** 9] * (steps - len(w)) for w in self.paths])      # behind the path: not read
        self.path_len = i32(self.sizes)
        self.k_out, self.v_out = (torch.full((self.B, self.L, steps, self.H, self.d), 3.0, dtype=torch.bfloat16,
                                             device="cuda").transpose(2, 3) for _ in range(2))
        used = torch.arange(self.rows.pos.shape[1], device="cuda") < self.rows.count[:, None]
        self.rows.mass.copy_(torch.where(used, torch.rand(used.shape, generator=self.g, device="cuda") * 3, self.rows.mass))

    def heads(self, b, l, h, x, kind):
        if kind == "q":
            return x[b, l, h * self.G:(h + 1) * self.G][:, self.paths[b]].double()
        return x[b, l, h][self.paths[b]].double()

    def commit(self, with_mass=True, scale=0.0, mods=None, **about):
        r = self.rows
        self.want, full = {}, 1 / math.sqrt(self.d) if not scale else scale
        slopes, prefix = about.get("slopes"), about.get("prefix", [-2 ** 40] * self.B)
        for b in range(self.B):
            for l in range(self.L):
                for h in range(self.H):
                    u = (b * self.L + l) * self.H + h
                    here = slice(h * self.G, h * self.G + self.G)
                    lse, w, e = path_mass(r, u, self.heads(b, l, h, self.q, "q"), self.heads(b, l, h, self.k, "k"), full,
                                          softcap=about.get("softcap", 0.0), window=about.get("window", 0), prefix=prefix[b],
                                          slopes=None if slopes is None else slopes[here]) if self.paths[b] else (None, None, None)
                    if lse is not None:
                        self.lse[b, l, here][:, self.paths[b]] = lse.float()
                    self.want[u] = (w, e)
        self.before = [t.clone() for t in fields(r)]
        self.again = lambda: kvc.kvc_i4_tree_commit(
            self.shape, r, self.k, self.v, self.path, self.path_len, q=self.q if with_mass else None,
            row_lse=self.lse if with_mass else None, mods=mods, softmax_scale=scale, k_out=self.k_out, v_out=self.v_out,
            unit_status=self.status)
        self.with_mass = with_mass
        self.again()
        return self

    def check_commit(self, left=()):
        """`left`: units that were to stay as they were."""
        torch.cuda.synchronize()
        r, was = self.rows, self.before
        for u in range(self.B * self.L * self.H):
            b, l, h = u // (self.L * self.H), u // self.H % self.L, u % self.H
            n, m = int(was[6][u]), len(self.paths[b])
            if u in left or m == 0:
                for t, t0 in zip(fields(r), was):
                    assert torch.equal(bits(t[u:u + 1]), bits(t0[u:u + 1])), u
                assert bool((self.k_out[b, l, h] == 3).all())
                continue
            assert int(r.count[u]) == n + m and int(r.next_pos[u]) == int(was[7][u]) + m
            new = slice(n, n + m)
            for x, codes, scale, out in ((self.k, r.k, r.k_scale, self.k_out), (self.v, r.v, r.v_scale, self.v_out)):
                want, s = o.quantize(x[b, l, h][self.paths[b]].float().cpu().numpy(), 7, r.quant_mode)
                assert np.array_equal(codes[u, new].cpu().numpy(), o.pack_int4(want))
                assert np.array_equal(scale[u, new].float().cpu().numpy(), s)
                assert torch.equal(out[b, l, h, :m], held(codes[u, new], scale[u, new], self.d).to(torch.bfloat16))
                assert bool((out[b, l, h, m:] == 3).all())
            assert torch.equal(r.pos[u, new], was[7][u] + torch.arange(m, device="cuda", dtype=torch.int32))
            for t, t0 in zip(fields(r)[:5], was[:5]):          # every other slot as it was
                assert torch.equal(bits(t[u, :n]), bits(t0[u, :n])) and torch.equal(bits(t[u, n + m:]), bits(t0[u, n + m:]))
            assert torch.equal(bits(r.mass[u, n + m:]), bits(was[5][u, n + m:]))
            if self.with_mass:
                w, e = self.want[u]
                old = torch.cat((was[5][u, :n].double(), torch.zeros(m, dtype=torch.float64, device="cuda")))
                close(r.mass[u, :n + m], old + w, e + 2 * U * (old + w), f"mass of unit {u}")
            else:
                assert torch.equal(r.mass[u, :n], was[5][u, :n]) and bool((r.mass[u, new] == 0).all())
        return self


@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,steps", [(1, 1), (4, 1), (4, 2), (3, 5), (4, 7), (8, 9)])
def test_paths(G, steps, d, mode):
    p = Commit(steps=steps, B=2, L=2, G=G, H=2, d=d, n=20, counts=(300, 129), spare=steps, mode=mode, kind="chain", seed=G)
    p.commit().check_commit()
    assert (p.status == 55).all()


@pytest.mark.parametrize("counts", [(0,), (1,), (31,), (32,), (33,), (127, 0, 128), (2304, 5), (20001, 300)], ids=str)
@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
def test_lengths(counts, mode):
    Commit(steps=3, B=len(counts), G=4, H=2, n=9, counts=counts, mode=mode).commit().check_commit()


@pytest.mark.parametrize("G,steps", [(4, 64), (1, 64), (33, 5)])
def test_long_paths(G, steps):
    Commit(steps=steps, B=1, G=G, H=2, d=64, n=64, counts=(500,), spare=64, kind="chain").commit().check_commit()


def test_strides():
    Commit(steps=4, B=3, L=2, G=3, H=2, n=21, counts=(140, 5, 333), spare=4, by_token=True).commit().check_commit()


def test_sequences_of_a_batch():
    """No node accepted, some, all that were asked for, and lengths outside the range."""
    p = Commit(steps=5, sizes=[0, 2, 5, -3], B=4, G=4, H=2, n=30, counts=(100, 90, 200, 64), spare=5)
    p.commit().check_commit()
    q = Commit(steps=3, B=1, G=2, H=1, n=9, counts=(50,), spare=3, kind="chain")
    q.path_len.fill_(99)                                       # limited to the path's columns
    q.commit().check_commit()


MODS = [dict(softcap=20.0), dict(softcap=1.0), dict(slopes=True), dict(window=1), dict(window=3), dict(window=130),
        dict(window=60, prefix=True), dict(softcap=30.0, slopes=True, window=500, prefix=True), dict(softcap=5000.0),
        dict(softcap=1e-30)]


@pytest.mark.parametrize("mods", MODS, ids=lambda m: "-".join(f"{k}{v}" for k, v in m.items()))
@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
def test_modifiers(mods, mode):
    p = Commit(steps=6, B=2, G=4, H=2, d=64, n=20, counts=(2700, 129), spare=6, mode=mode, kind="chain", seed=3)
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(8)], device="cuda") if mods.get("slopes") else None
    prefix = [90, 3] if mods.get("prefix") else [0, 0]
    m = kvc.ScoreMods(mods.get("softcap", 0.0), slopes, mods.get("window", 0), i32(prefix) if mods.get("prefix") else None)
    p.commit(mods=m, softcap=mods.get("softcap", 0.0), slopes=slopes, window=mods.get("window", 0), prefix=prefix).check_commit()


def test_without_queries_and_without_mass():
    p = Commit(steps=3, B=1, G=4, H=2, n=9, counts=(70,)).commit(with_mass=False).check_commit()
    before = [t.clone() for t in fields(p.rows)]
    q = Commit(steps=3, B=1, G=4, H=2, n=9, counts=(70,))
    q.rows.mass = None
    kvc.kvc_i4_tree_commit(q.shape, q.rows, q.k, q.v, q.path, q.path_len)
    torch.cuda.synchronize()
    for name in ("k", "pos", "count", "next_pos"):
        assert torch.equal(getattr(q.rows, name), getattr(p.rows, name))
    assert len(before) == 8


@pytest.mark.parametrize("nxt", [2 ** 31 - 30, 0, -2 ** 31 + 2000])
def test_positions_over_all_of_int32(nxt):
    for about in (dict(window=250), dict(slopes=torch.full((8,), 2.0 ** -30, device="cuda"))):
        p = Commit(steps=4, B=1, G=4, H=2, n=20, counts=(700,), spare=4, kind="chain", seed=6)
        pos = torch.randint(-2 ** 31, nxt, (2, 700), generator=gen(3), device="cuda")
        pos[:, :300] = nxt - 1 - torch.arange(300, device="cuda")
        pos[:, 300] = -2 ** 31
        p.rows.pos[:, :700] = pos.to(torch.int32)
        p.rows.next_pos.fill_(nxt)
        p.commit(mods=kvc.ScoreMods(0.0, about.get("slopes"), about.get("window", 0)), **about).check_commit()


@pytest.mark.parametrize("G,steps,window", [(1, 3, 0), (4, 4, 0), (4, 3, 200)])
def test_statistics_of_rows_that_saw_nothing(G, steps, window):
    """Such a row has no weights, whatever its scores: the second node's rows are those."""
    p = Commit(steps=steps, B=1, G=G, H=2, n=9, counts=(150,), spare=steps, kind="chain")
    mods = kvc.ScoreMods(window=window) if window else None
    p.commit(mods=mods, window=window)
    kept = p.rows.mass.clone()
    p.lse[:, :, :, p.paths[0][1]] = -math.inf
    for x, x0 in zip(fields(p.rows), p.before):
        x.copy_(x0)
    p.again()
    torch.cuda.synchronize()
    used = slice(0, 150 + steps)
    now = p.rows.mass[:, used]
    assert bool(torch.isfinite(now).all()) and bool((now <= kept[:, used]).all())
    # less by the weights of G rows
    lost = (kept[:, used] - now).double().sum(1)
    assert bool(((lost - G).abs() < 1e-3 * G).all())


def test_nothing_accepted_then_more():
    """A step that accepts nothing, with calls in front of and behind it in the stream."""
    p = Commit(steps=3, sizes=[0, 0], B=2, G=4, H=2, n=9, counts=(500, 300), spare=8)
    p.commit().check_commit()
    for _ in range(4):
        p.again()
        kvc.kvc_i4_append(p.shape, p.rows, p.k[:, :, :, :1], p.v[:, :, :, :1])
    torch.cuda.synchronize()
    assert p.rows.count.tolist() == [504, 504, 304, 304]


def test_scale():
    Commit(steps=3, n=9, spare=3).commit(scale=0.37).check_commit()


def test_what_does_not_fit_or_is_no_node_changes_nothing():
    p = Commit(steps=3, B=6, G=2, H=1, n=9, counts=(50, 48, 47, 20, 20, 20), spare=0)
    for u, c in ((0, 50), (1, 48), (2, 47), (5, -1)):
        p.rows.count[u] = c
    p.path[3, 1], p.path[4, 0] = 9, -1
    p.paths[5] = []                                            # (its weights are not formed here: the count is no count)
    p.commit().check_commit(left=(0, 1, 3, 4, 5))
    full, bad = kvc.UNIT_FULL, kvc.UNIT_BAD_INDEX
    assert p.status.tolist() == [full, full, 55, bad, bad, bad]


def test_repeats_graphs_and_streams():
    p = Commit(steps=4, B=2, G=4, H=2, n=17, counts=(3000, 1200), spare=50, kind="chain").commit().check_commit()
    first = [t.clone() for t in fields(p.rows)]
    for t, t0 in zip(fields(p.rows), p.before):
        t.copy_(t0)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.again()
    side.synchronize()
    assert all(torch.equal(bits(t), bits(t0)) for t, t0 in zip(fields(p.rows), first))
    with torch.cuda.graph(graph):
        p.again()
    for t, t0 in zip(fields(p.rows), p.before):
        t.copy_(t0)
    graph.replay()
    p.check_commit()
    for _ in range(3):                                         # the same path again, behind itself
        graph.replay()
    torch.cuda.synchronize()
    assert p.rows.count.tolist() == [3016, 3016, 1216, 1216]
    assert torch.equal(p.rows.pos[0, 3012:3016], p.rows.pos[0, 3000:3004] + 12)


def test_rows_past_32_bit_offsets():
    """A cache of 40 units of 900,000 rows, the last of them committed to (2.3e9 bytes of codes in front of it)."""
    units, cap, d = 40, 900_000, 128
    shape = kvc.make_shape(1, units, 1, 1, d, 1)
    rows = kvc.I4Rows.allocate(shape, cap)
    p = Commit(steps=3, B=1, L=1, G=1, H=1, d=d, n=5, counts=(500,), spare=3, kind="chain")
    for name in ("k", "v", "k_scale", "v_scale", "pos", "mass"):
        getattr(rows, name)[units - 1, :503] = getattr(p.rows, name)[0, :503]
    rows.count[units - 1] = 500
    rows.next_pos[units - 1] = p.rows.next_pos[0]
    p.commit()
    q, k, v = (torch.zeros(1, units, 1, 5, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    q[0, units - 1], k[0, units - 1], v[0, units - 1] = p.q[0, 0], p.k[0, 0], p.v[0, 0]
    lse = torch.zeros(1, units, 1, 5, device="cuda")
    lse[0, units - 1] = p.lse[0, 0]
    kvc.kvc_i4_tree_commit(shape, rows, k, v, p.path, p.path_len, q=q, row_lse=lse)
    torch.cuda.synchronize()
    for name in ("k", "v", "k_scale", "v_scale", "pos"):
        assert torch.equal(bits(getattr(rows, name)[units - 1, :503]), bits(getattr(p.rows, name)[0, :503]))
    p.rows.mass[0, :503] = rows.mass[units - 1, :503]
    p.check_commit()


@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
def test_drafting_over_a_budgeted_cache(mode):
    """Steps of a program: new tokens rotated, a tree checked, its accepted path committed, the rows of least mass evicted.
    Each call is checked from the state that the one before it left."""
    B, G, H, d, n, steps, budget = 2, 4, 2, 128, 24, 5, 256
    p = Commit(steps=steps, B=B, G=G, H=H, d=d, n=n, counts=(budget, 200), spare=steps, mode=mode, seed=2)
    cos, sin = torch.empty(4096, d // 2, device="cuda"), torch.empty(4096, d // 2, device="cuda")
    kvc.kvc_rope_tables(cos, sin, 10000.0, kvc.RopeScaling(kvc.ROPE_SCALE_LINEAR, 2.0))
    ws = torch.empty(max(256, kvc.kvc_i4_evict_workspace_bytes(p.shape, p.rows, budget)), dtype=torch.uint8, device="cuda")
    for step in range(4):
        g = gen(50 + step)
        p.parents = [trees("random", n, 10 * step + b) for b in range(B)]
        p.parent.copy_(i32(p.parents))
        for t, size in ((p.q, 2.0), (p.k, 1.0), (p.v, 1.0)):
            t.copy_(randn(g, *t.shape) * size)
        nxt = p.rows.next_pos.view(B, H)[:, 0].tolist()
        pos = i32([[nxt[b] + len(w) - 1 for w in lines(p.parents[b])] for b in range(B)])
        kvc.kvc_rope(p.shape, p.q, p.k, pos, cos, sin)
        p.out.fill_(7)
        p.lse.fill_(7)
        p.status.fill_(55)
        p.call().check()
        p.paths = [max(lines(p.parents[b]), key=len)[:1 + (step + b) % steps] for b in range(B)]
        p.path.copy_(i32([w + [0] * (steps - len(w)) for w in p.paths]))
        p.path_len.copy_(i32([len(w) for w in p.paths]))
        p.k_out.fill_(3)
        p.v_out.fill_(3)
        mine = p.lse.clone()                                   # the attention's own statistics
        p.commit()
        torch.cuda.synchronize()
        for b in range(B):
            assert float((mine[b][..., p.paths[b]] - p.lse[b][..., p.paths[b]]).abs().max()) < 1e-5
        p.check_commit()
        kvc.kvc_i4_evict(p.shape, p.rows, budget, 4, 16, workspace=ws)
        torch.cuda.synchronize()
        assert int(p.rows.count.max()) <= budget
