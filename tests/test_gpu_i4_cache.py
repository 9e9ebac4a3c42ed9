"""The growing 4-bit cache against the oracle's quantiser and 64-bit definitions: append and read (codes,
scales, positions, counters, overflow), attention with accumulated mass, eviction in place, and a prompt and
its tokens run through all of them."""
import math
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import oracle as o
from attn_reference import attend, close, visible

pytestmark = pytest.mark.gpu

G32, ROW = 0, 1


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()
    import budgeted_kv_cache_gb300 as lib
    lib.library()
    return lib


def gen(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *s):
    return torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def held(codes, scale, d):
    """64-bit values of packed rows."""
    c = torch.from_numpy(o.unpack_int4(codes.cpu().numpy()).astype(np.float64)).to(codes.device)
    return c * scale.double().repeat_interleave(d // scale.shape[-1], -1)


def fields(rows):
    return [rows.k, rows.v, rows.k_scale, rows.v_scale, rows.pos, rows.mass, rows.count, rows.next_pos]


def snapshot(rows):
    return [t.clone() for t in fields(rows)]


def scramble(rows, g):
    """Garbage in every row (also scales of NaN), as in memory that was used before."""
    for t in (rows.k, rows.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (rows.k_scale, rows.v_scale, rows.mass):
        t.fill_(float("nan"))
    rows.pos.fill_(-7)


# ---------------------------------------------------------------- append, read

@pytest.mark.parametrize("mode", [G32, ROW], ids=["g32", "row"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 17, 255, 257, 1500])
def test_append_and_read(kvc, n, d, mode):
    B, L, H, cap = 2, 2, 3, n + 5
    shape, g = kvc.make_shape(B, L, H, H, d, 1), gen(n)
    rows = kvc.I4Rows.allocate(shape, cap, mode)
    scramble(rows, g)
    U = B * L * H
    rows.count.copy_(torch.randint(0, 6, (U,), generator=g, device="cuda"))
    rows.next_pos.copy_(torch.randint(0, 100, (U,), generator=g, device="cuda"))
    k, v = randn(g, B, L, n, H, d).transpose(2, 3), randn(g, B, L, n, H, d).transpose(2, 3)
    k[0, 0, 0, 0] = 0                                          # a zero row
    k[0, 0, 1, 0, :32] *= 2.0 ** -120                          # scales at the formats' ends
    v[0, 0, 1, 0] *= 2.0 ** (100 if mode == G32 else -30)
    v[1, 1, 2, n - 1] = torch.arange(d, device="cuda").to(torch.bfloat16) / 2    # ties of the rounding
    n_new = [n, n // 2]
    before = snapshot(rows)
    kvc.kvc_i4_append(shape, rows, k, v, n_new=i32(n_new))
    torch.cuda.synchronize()
    for u in range(U):
        m, c0 = n_new[u // (L * H)], int(before[6][u])
        assert int(rows.count[u]) == c0 + m and int(rows.next_pos[u]) == int(before[7][u]) + m
        new = slice(c0, c0 + m)
        for x, codes, scale in ((k, rows.k, rows.k_scale), (v, rows.v, rows.v_scale)):
            xu = x[u // (L * H), u // H % L, u % H, :m].float().cpu().numpy()
            want, s = o.quantize(xu, 7, mode)
            assert np.array_equal(codes[u, new].cpu().numpy(), o.pack_int4(want))
            assert np.array_equal(scale[u, new].float().cpu().numpy(), s)
        assert torch.equal(rows.pos[u, new], before[7][u] + torch.arange(m, device="cuda", dtype=torch.int32))
        assert bool((rows.mass[u, new] == 0).all())
        for t, t0 in zip(fields(rows)[:6], before[:6]):        # every other slot as it was
            keep = torch.ones(cap, dtype=torch.bool, device="cuda")
            keep[new] = False
            assert torch.equal(t[u, keep].contiguous().view(torch.uint8), t0[u, keep].contiguous().view(torch.uint8))
    # read back: code * scale rounded once; rows that are not in use stay
    k_out, v_out = (torch.full((B, L, cap, H, d), 3.0, dtype=torch.bfloat16, device="cuda").transpose(2, 3) for _ in range(2))
    kvc.kvc_i4_read(shape, rows, k_out, v_out)
    torch.cuda.synchronize()
    for u in range(U):
        c = int(rows.count[u])
        lo = int(before[6][u])
        for out, codes, scale in ((k_out, rows.k, rows.k_scale), (v_out, rows.v, rows.v_scale)):
            got = out[u // (L * H), u // H % L, u % H]
            want = held(codes[u, lo:c], scale[u, lo:c], d).to(torch.bfloat16)
            assert torch.equal(got[lo:c], want)
            assert bool((got[c:] == 3).all())


def test_append_that_does_not_fit_changes_nothing(kvc):
    shape, g = kvc.make_shape(4, 1, 1, 1, 64, 1), gen(1)
    rows = kvc.I4Rows.allocate(shape, 300)
    scramble(rows, g)
    rows.count.copy_(i32([0, 20, 21, -1]))
    before = snapshot(rows)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    kvc.kvc_i4_append(shape, rows, randn(g, 4, 1, 1, 280, 64), randn(g, 4, 1, 1, 280, 64), unit_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0, kvc.UNIT_FULL, kvc.UNIT_BAD_INDEX]
    assert rows.count.tolist() == [280, 300, 21, -1]
    for t, t0 in zip(fields(rows), before):
        assert torch.equal(t[2:].contiguous().view(torch.uint8), t0[2:].contiguous().view(torch.uint8))


def test_appending_nothing(kvc):
    shape, g = kvc.make_shape(2, 1, 1, 1, 64, 1), gen(1)
    rows = kvc.I4Rows.allocate(shape, 8)
    scramble(rows, g)
    before = snapshot(rows)
    x = randn(g, 2, 1, 1, 3, 64)
    kvc.kvc_i4_append(shape, rows, x, x, n_new=i32([0, -4]))
    kvc.kvc_i4_append(shape, rows, x[:, :, :, :0], x[:, :, :, :0])
    kvc.kvc_i4_read(shape, rows, x[:, :, :, :0], x[:, :, :, :0])
    torch.cuda.synchronize()
    for t, t0 in zip(fields(rows), before):
        assert torch.equal(t.contiguous().view(torch.uint8), t0.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- attention

class Cache:
    """A cache as eviction leaves it: positions with gaps in any slot order, garbage behind the rows in use."""

    def __init__(self, kvc, B, L, Hkv, d, cap, counts, mode, seed=0, n_q_heads=None):
        g = gen(seed)
        self.kvc, self.g, self.d = kvc, g, d
        self.shape = kvc.make_shape(B, L, n_q_heads or Hkv, Hkv, d, 1)
        U = B * L * Hkv
        full = kvc.I4Rows.allocate(self.shape, cap, mode)
        kvc.kvc_i4_append(self.shape, full, randn(g, B, L, Hkv, cap, d), randn(g, B, L, Hkv, cap, d))
        torch.cuda.synchronize()
        rows = self.rows = full
        gaps = torch.cumsum(torch.randint(1, 4, (U, cap), generator=g, device="cuda"), 1)
        order = torch.argsort(torch.rand(U, cap, generator=g, device="cuda"), 1)
        rows.pos.copy_(gaps.gather(1, order))
        rows.mass.copy_(torch.rand(U, cap, generator=g, device="cuda"))
        rows.count.copy_(i32(counts).repeat_interleave(U // len(counts)))
        rows.next_pos.copy_(gaps[:, -1] + 1)
        behind = torch.arange(cap, device="cuda") >= rows.count[:, None]
        for t in (rows.k_scale, rows.v_scale):
            t.masked_fill_(behind[..., None], float("nan"))


def check_attention(c, q, out, lse, mass0, q_pos=None, softcap=0.0, slopes=None, window=0, prefix=None, add=False,
                    scale=0.0):
    torch.cuda.synchronize()
    r, s = c.rows, c.shape
    G = s.n_q_heads // s.n_kv_heads
    scale = scale or 1 / math.sqrt(c.d)
    n_q = q.shape[3]
    for u in range(s.batch * s.n_layers * s.n_kv_heads):
        b, l, h0 = u // (s.n_layers * s.n_kv_heads), u // s.n_kv_heads % s.n_layers, u % s.n_kv_heads
        n = max(0, min(int(r.count[u]), r.pos.shape[1]))
        k, v = held(r.k[u, :n], r.k_scale[u, :n], c.d), held(r.v[u, :n], r.v_scale[u, :n], c.d)
        p_q = (int(r.next_pos[u]) - n_q + torch.arange(n_q, device="cuda")) if q_pos is None else q_pos[b].long()
        p_k = r.pos[u, :n].long()
        seen = visible(p_q, p_k, window, -(1 << 40) if prefix is None else int(prefix[b]))
        dist = (p_q[:, None] - p_k[None]).double()
        add_w, add_e = torch.zeros(n, device="cuda", dtype=torch.float64), torch.zeros(n, device="cuda", dtype=torch.float64)
        for h in range(h0 * G, h0 * G + G):
            want, wl, w, e_o, e_l, e_w = attend(q[b, l, h].double(), k, v, scale, seen, dist, softcap,
                                                None if slopes is None else float(slopes[h]))
            close(out[b, l, h], want, e_o, f"out u{u} h{h}")
            close(lse[b, l, h], wl, e_l, f"lse u{u} h{h}")
            add_w += w.sum(0)
            add_e += e_w.sum(0) + G * n_q * 2.0 ** -24 * w.sum(0)
        want = mass0[u].double().clone()
        bound = torch.zeros_like(want)
        if add:
            want[:n] += add_w
            bound[:n] = add_e + 2.0 ** -24 * want[:n]
        close(r.mass[u], want, bound, f"mass u{u}")


ATTN = {
    "one_row": dict(cap=1, counts=[1]),
    "no_rows": dict(B=2, cap=40, counts=[0, 40]),
    "counts_out_of_range": dict(B=2, cap=40, counts=[-5, 41]),
    "odd": dict(B=2, L=2, Hkv=2, G=4, cap=133, counts=[133, 50], add=True),
    "tile_edge": dict(B=3, cap=256, counts=[64, 128, 129], add=True),
    "long": dict(Hkv=2, G=4, cap=9001, counts=[9001], add=True),
    "long_row_mode": dict(Hkv=1, G=8, d=64, cap=7777, counts=[7000], mode=ROW, add=True),
    "one_head": dict(Hkv=3, G=1, cap=700, counts=[700], add=True),
    "three_heads": dict(Hkv=2, G=3, cap=700, counts=[699], d=64, add=True),
    "seven_heads": dict(Hkv=1, G=7, cap=700, counts=[650], mode=ROW, add=True),
    "wide_group": dict(Hkv=1, G=33, cap=500, counts=[500], add=True),
    "draft": dict(B=2, Hkv=2, G=4, n_q=5, cap=800, counts=[800, 3], add=True),
    "chunk": dict(B=1, Hkv=1, G=4, n_q=70, cap=900, counts=[900], add=True),
    "many_units": dict(B=5, L=7, Hkv=9, G=1, cap=40, counts=[40, 0, 33, 1, 32], add=True),
    "chunk_d64": dict(B=2, Hkv=2, G=2, n_q=33, cap=300, counts=[300, 128], d=64, mode=ROW),
    "softcap": dict(Hkv=2, G=4, n_q=3, cap=600, counts=[600], softcap=4.0, q_norm=8.0, add=True),
    "slopes": dict(Hkv=2, G=4, n_q=2, cap=600, counts=[600], slopes=True, add=True),
    "window": dict(Hkv=2, G=4, n_q=4, cap=900, counts=[900], window=100, add=True),
    "window_nothing": dict(Hkv=1, G=2, n_q=2, cap=90, counts=[20], window=1, add=True),
    "prefix": dict(B=2, Hkv=1, G=2, n_q=4, cap=500, counts=[500, 400], window=30, prefix=[200, 0], add=True),
    "window_many_rows": dict(Hkv=1, G=5, n_q=11, cap=2000, counts=[1900], window=40, add=True),
    "given_positions": dict(B=2, Hkv=2, G=2, n_q=3, cap=300, counts=[300, 200], q_pos=[[-1, 100, 5000], [0, 7, 200]], add=True),
    "everything": dict(B=2, L=2, Hkv=2, G=5, n_q=7, cap=1500, counts=[1500, 700], softcap=8.0, slopes=True, window=900,
                       prefix=[50, 0], add=True, token=True),
    "own_scale": dict(Hkv=1, G=4, cap=300, counts=[300], scale=0.3),
}


def attention_case(kvc, B=1, L=1, Hkv=1, G=4, d=128, cap=1, counts=(1,), mode=G32, n_q=1, softcap=0.0, slopes=False,
                   window=0, prefix=None, q_pos=None, add=False, q_norm=2.0, scale=0.0, token=False, seed=0):
    c = Cache(kvc, B, L, Hkv, d, cap, list(counts), mode, seed, Hkv * G)
    q = randn(c.g, B, L, n_q, Hkv * G, d).transpose(2, 3) if token else randn(c.g, B, L, Hkv * G, n_q, d)
    q.mul_(q_norm)
    sl = torch.rand(Hkv * G, generator=c.g, device="cuda") * 0.01 if slopes else None
    pre, qp = None if prefix is None else i32(prefix), None if q_pos is None else i32(q_pos)
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:-1], 9.0, device="cuda")
    ws = torch.empty(max(1, kvc.kvc_i4_attn_workspace_bytes(c.shape, c.rows, n_q, add)), dtype=torch.uint8, device="cuda")

    def run(stream=None):
        kvc.kvc_i4_attn(c.shape, c.rows, q, out, q_pos=qp, mods=kvc.ScoreMods(softcap, sl, window, pre),
                        softmax_scale=scale, add_mass=add, row_lse=lse, workspace=ws, stream=stream)
    check = lambda mass0: check_attention(c, q, out, lse, mass0, qp, softcap, sl, window, pre, add, scale)
    return c, run, check, out, lse


@pytest.mark.parametrize("name", ATTN)
def test_attention_matches_the_definition(kvc, name):
    c, run, check, _, _ = attention_case(kvc, **ATTN[name])
    mass0 = c.rows.mass.clone()
    run()
    check(mass0)


def test_attention_same_bits_twice_and_on_another_stream(kvc):
    c, run, check, out, lse = attention_case(kvc, **ATTN["long"])
    mass0 = c.rows.mass.clone()
    got = []
    s = torch.cuda.Stream()
    for stream in (None, s):
        c.rows.mass.copy_(mass0)
        out.zero_()
        s.wait_stream(torch.cuda.current_stream())
        run(stream)
        torch.cuda.synchronize()
        got.append((out.clone(), lse.clone(), c.rows.mass.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_attention_on_two_streams_at_once(kvc):
    """Calls that overlap over caches and workspaces of their own."""
    cases = [attention_case(kvc, Hkv=2, G=4, cap=6000, counts=[6000], add=True, seed=s) for s in (1, 2)]
    before = [c[0].rows.mass.clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c, s in zip(cases, streams):
        c[1](s)
    torch.cuda.synchronize()
    for c, m in zip(cases, before):
        c[2](m)


def test_mass_of_several_calls_adds_up(kvc):
    c, run, check, _, _ = attention_case(kvc, Hkv=2, G=4, cap=700, counts=[700], add=True)
    run()
    torch.cuda.synchronize()
    after_one = c.rows.mass.clone()
    run()
    check(after_one)


def test_attention_extreme_scales(kvc):
    """Value scales over the whole range of bf16: the weights carry them, and nothing overflows that the result does not."""
    c, run, check, _, _ = attention_case(kvc, Hkv=2, G=4, cap=300, counts=[300], add=True)
    e = torch.randint(-100, 30, c.rows.v_scale.shape, generator=c.g, device="cuda")
    c.rows.v_scale.copy_(torch.exp2(e.float()))
    c.rows.k_scale.mul_(torch.exp2(torch.randint(-60, 1, c.rows.k_scale.shape, generator=c.g, device="cuda").float()))
    mass0 = c.rows.mass.clone()
    run()
    check(mass0)


def test_attention_without_mass_array(kvc):
    c, run, check, out, lse = attention_case(kvc, Hkv=1, G=2, cap=50, counts=[50])
    mass = c.rows.mass
    c.rows.mass = None
    run()
    c.rows.mass = mass
    check(mass)
    c.rows.mass = None
    with pytest.raises(kvc.KvcError):
        kvc.kvc_i4_attn(c.shape, c.rows, out.clone(), out, add_mass=True,
                        workspace=torch.empty(1 << 16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kvc.KvcError):
        kvc.kvc_i4_evict(c.shape, c.rows, 8, 0, 0, workspace=torch.empty(1 << 16, dtype=torch.uint8, device="cuda"))


def test_compaction_pools_as_a_growing_cache(kvc):
    """The int4 pool of a byte-mode compaction attended as it is."""
    import workloads as wl
    from budgeted_kv_cache_gb300.passes import pass_for_workload
    w = wl.pask_batch16().replace(name="i4_pools", batch=2, n_layers=4, n_kv_heads=2, n_q_heads=8, n_tokens=900, window=16,
                                  n_recent=16, budget_bytes=(900 * 512) // 3, decode_pos=900)
    x = wl.make_inputs(w, "cuda")
    p = pass_for_workload(w, inputs=x)
    p.run(x["k_cache"], x["v_cache"], x["q_window"], x["pos_in"], x["rope_cos"], x["rope_sin"], x.get("bonus"))
    torch.cuda.synchronize()
    U = w.n_units
    c = Cache.__new__(Cache)
    c.kvc, c.shape, c.d = kvc, p.shape, w.head_dim
    nxt = torch.full((U,), 900, dtype=torch.int32, device="cuda")
    cap = p.pools.pos_out.shape[2]
    c.rows = kvc.I4Rows.from_pools(p.pools, p.policy, p.kept_count, nxt, torch.zeros(U, cap, device="cuda"))
    assert int(c.rows.count.max()) > 0
    q = randn(gen(2), w.batch, w.n_layers, w.n_q_heads, 1, w.head_dim)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:-1], device="cuda")
    ws = torch.empty(max(1, kvc.kvc_i4_attn_workspace_bytes(c.shape, c.rows, 1, True)), dtype=torch.uint8, device="cuda")
    kvc.kvc_i4_attn(c.shape, c.rows, q, out, add_mass=True, row_lse=lse, workspace=ws)
    check_attention(c, q, out, lse, torch.zeros(U, cap, device="cuda"), add=True)


# ---------------------------------------------------------------- eviction

def evicted(pos, mass, cnt, nxt, budget, n_sink, n_recent):
    """Source slot of each kept slot, or a status, from the definition."""
    over = cnt - budget
    if over <= 0:
        return np.arange(cnt), 0
    m = np.where(np.isnan(mass), -np.inf, mass)
    free = [i for i in range(cnt) if n_sink <= pos[i] < nxt - n_recent]
    if len(free) < over:
        return np.arange(cnt), 1
    gone = set(sorted(free, key=lambda i: (m[i], -int(pos[i]), i))[:over])
    donors = iter([i for i in range(budget, cnt) if i not in gone])
    return np.array([next(donors) if i in gone else i for i in range(budget)]), 0


EVICT = {
    "one": dict(cap=65, counts=[65], budget=64),
    "many": dict(cap=700, counts=[700], budget=200),
    "long": dict(cap=20000, counts=[20000], budget=2048, U=2),
    "long_few": dict(cap=33000, counts=[33000], budget=32990, U=2),
    "ragged": dict(cap=300, counts=[300, 100, 101, 0, 299], budget=100),
    "ties": dict(cap=500, counts=[500], budget=123, ties=True),
    "all_equal": dict(cap=300, counts=[300], budget=77, equal=True),
    "nan_and_zeros": dict(cap=300, counts=[300], budget=200, odd_values=True),
    "over_budget": dict(cap=200, counts=[200, 150], budget=100, n_recent=400),
    "no_protection": dict(cap=100, counts=[100], budget=1, n_sink=0, n_recent=0),
    "counts_out_of_range": dict(cap=100, counts=[101, -1, 100], budget=50),
    "budget_over_capacity": dict(cap=100, counts=[100], budget=1000),
    "same_positions": dict(cap=200, counts=[200], budget=90, same=True, equal=True),
    "every_row_but_one_leaves": dict(cap=3000, counts=[3000], budget=1, n_sink=0, n_recent=1, U=2),
    "more_moves_than_shared": dict(cap=9000, counts=[9000], budget=4500, U=2),
    "more_words_than_shared": dict(cap=40000, counts=[40000], budget=39000, U=1, ties=True),
    "row_mode": dict(cap=400, counts=[400], budget=300, mode=ROW),
    "d64": dict(cap=400, counts=[400], budget=300, d=64),
}


@pytest.mark.parametrize("name", EVICT)
def test_evict(kvc, name):
    kw = dict(EVICT[name])
    cap, counts, budget = kw["cap"], kw["counts"], kw["budget"]
    B, U, d, mode = len(counts), kw.get("U", 3), kw.get("d", 128), kw.get("mode", G32)
    n_sink, n_recent = kw.get("n_sink", 4), kw.get("n_recent", 16)
    c = Cache(kvc, B, 1, U, d, cap, counts, mode, seed=4)
    r, status = c.rows, torch.zeros(B * U, dtype=torch.int32, device="cuda")
    if kw.get("ties"):
        r.mass.mul_(8).floor_()
    if kw.get("equal"):
        r.mass.fill_(0.5)
    if kw.get("odd_values"):
        r.mass[:, ::3], r.mass[:, 1::7], r.mass[:, 2::5] = float("nan"), -0.0, 0.0
        r.mass[:, 4::11], r.mass[:, 5::13] = float("inf"), -1.0
    if kw.get("same"):
        r.pos.fill_(50)
        r.next_pos.fill_(500)
    before = snapshot(r)
    ws = torch.empty(max(1, kvc.kvc_i4_evict_workspace_bytes(c.shape, r, budget)), dtype=torch.uint8, device="cuda")
    kvc.kvc_i4_evict(c.shape, r, budget, n_sink, n_recent, unit_status=status, workspace=ws)
    torch.cuda.synchronize()
    b_pos, b_mass = before[4].cpu().numpy(), before[5].cpu().numpy()
    for u in range(B * U):
        cnt = int(before[6][u])
        if not 0 <= cnt <= cap:
            src, want, n = np.arange(cap), kvc.UNIT_BAD_INDEX, cnt
        else:
            src, st = evicted(b_pos[u], b_mass[u], cnt, int(before[7][u]), budget, n_sink, n_recent)
            want, n = (kvc.UNIT_OVER_BUDGET, cnt) if st else (0, len(src))
            src = np.concatenate([src, np.arange(len(src), cap)])
        assert int(status[u]) == want and int(r.count[u]) == n
        at = torch.from_numpy(src).cuda()
        for t, t0 in zip(fields(r)[:6], before[:6]):
            assert torch.equal(t[u].contiguous().view(torch.uint8), t0[u][at].contiguous().view(torch.uint8))
        assert int(r.next_pos[u]) == int(before[7][u])


# ---------------------------------------------------------------- large caches

def test_more_units_than_a_grid_dimension_holds(kvc):
    """2 x 32,800 units in one call: the bits of a call for each half."""
    B, H, d, cap = 2, 32800, 64, 4
    g = gen(9)
    k, v, q = randn(g, B, 1, H, 3, d), randn(g, B, 1, H, 3, d), randn(g, B, 1, H, 1, d)

    def run(b0, b1):
        n = b1 - b0
        shape = kvc.make_shape(n, 1, H, H, d, 1)
        rows = kvc.I4Rows.allocate(shape, cap)
        for t in fields(rows)[:6]:
            t.zero_()
        out, lse = torch.empty_like(q[b0:b1]), torch.empty(n, 1, H, 1, device="cuda")
        k_out, v_out = torch.zeros_like(k[b0:b1]), torch.zeros_like(k[b0:b1])
        kvc.kvc_i4_append(shape, rows, k[b0:b1], v[b0:b1])
        ws = torch.empty(kvc.kvc_i4_attn_workspace_bytes(shape, rows, 1, True), dtype=torch.uint8, device="cuda")
        kvc.kvc_i4_attn(shape, rows, q[b0:b1], out, add_mass=True, row_lse=lse, workspace=ws)
        ws = torch.empty(max(1, kvc.kvc_i4_evict_workspace_bytes(shape, rows, 2)), dtype=torch.uint8, device="cuda")
        kvc.kvc_i4_evict(shape, rows, 2, 0, 0, workspace=ws)
        kvc.kvc_i4_read(shape, rows, k_out, v_out)
        torch.cuda.synchronize()
        assert bool((rows.count == 2).all()) and bool((rows.next_pos == 3).all())
        return [out, lse, k_out, v_out] + fields(rows)

    for whole, first, second in zip(run(0, 2), run(0, 1), run(1, 2)):
        assert torch.equal(whole, torch.cat([first, second]))


def test_rows_past_32_bit_offsets(kvc):
    """Units of 70 million slots: the second one's rows lie past 2^31 bytes."""
    small, n = Cache(kvc, 1, 1, 2, 64, 320, [300], ROW, n_q_heads=4), 320
    big = kvc.I4Rows.allocate(small.shape, 70_000_000, ROW)
    part = [t[:, :n] if t.dim() > 1 else t for t in fields(big)]
    for t, t0 in zip(part, fields(small.rows)):
        t.copy_(t0)
    x, y, q = randn(small.g, 1, 1, 2, 10, 64), randn(small.g, 1, 1, 2, 10, 64), randn(small.g, 1, 1, 4, 2, 64)
    for rows in (small.rows, big):
        kvc.kvc_i4_append(small.shape, rows, x, y)
    torch.cuda.synchronize()
    for t, t0 in zip(part, fields(small.rows)):
        assert torch.equal(t.contiguous().view(torch.uint8), t0.contiguous().view(torch.uint8))
    out, lse, mass0 = torch.empty_like(q), torch.empty(q.shape[:-1], device="cuda"), part[5].clone()
    ws = torch.empty(kvc.kvc_i4_attn_workspace_bytes(small.shape, big, 2, True), dtype=torch.uint8, device="cuda")
    kvc.kvc_i4_attn(small.shape, big, q, out, add_mass=True, row_lse=lse, workspace=ws)
    names = ["k", "v", "k_scale", "v_scale", "pos", "mass", "count", "next_pos"]
    check_attention(SimpleNamespace(rows=SimpleNamespace(**dict(zip(names, part))), shape=small.shape, d=64), q, out, lse,
                    mass0, add=True)
    small.rows.mass.copy_(part[5])
    outs = []
    for rows in (small.rows, big):
        ws = torch.empty(max(1, kvc.kvc_i4_evict_workspace_bytes(small.shape, rows, 305)), dtype=torch.uint8, device="cuda")
        kvc.kvc_i4_evict(small.shape, rows, 305, 4, 16, workspace=ws)
        outs.append([torch.zeros(1, 1, 2, n, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)])
        kvc.kvc_i4_read(small.shape, rows, *outs[-1])
    torch.cuda.synchronize()
    assert big.count.tolist() == [305, 305]
    for t, t0 in zip(part + outs[1], fields(small.rows) + outs[0]):
        assert torch.equal(t.contiguous().view(torch.uint8), t0.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_prompt_then_tokens(kvc, graph):
    """A prompt is attended and stored; then per token: append, attend with mass, evict.  Every step's
    attention is checked over the rows that the cache then holds; positions stay those of the tokens."""
    B, L, Hkv, G, d, T, budget, steps = 2, 2, 2, 4, 128, 300, 256, 12
    g = gen(9)
    shape = kvc.make_shape(B, L, Hkv * G, Hkv, d, T)
    q, k, v = randn(g, B, L, Hkv * G, T, d), randn(g, B, L, Hkv, T, d), randn(g, B, L, Hkv, T, d)
    lens = i32([300, 260])
    po = torch.zeros_like(q)
    ws = torch.empty(max(256, kvc.kvc_prompt_attn_workspace_bytes(shape, T)), dtype=torch.uint8, device="cuda")
    kvc.kvc_prompt_attn(shape, q, k, v, po, q_len=lens, kv_len=lens, workspace=ws)
    rows = kvc.I4Rows.allocate(shape, T + 4)
    rows.mass.zero_()
    kvc.kvc_i4_append(shape, rows, k, v, n_new=lens)
    c = Cache.__new__(Cache)
    c.kvc, c.shape, c.d, c.rows = kvc, shape, d, rows
    aw = torch.empty(max(256, kvc.kvc_i4_attn_workspace_bytes(shape, rows, 1, True)), dtype=torch.uint8, device="cuda")
    ew = torch.empty(max(256, kvc.kvc_i4_evict_workspace_bytes(shape, rows, budget)), dtype=torch.uint8, device="cuda")
    tq, tk, tv = randn(g, B, L, Hkv * G, 1, d), randn(g, B, L, Hkv, 1, d), randn(g, B, L, Hkv, 1, d)
    out, lse = torch.empty_like(tq), torch.empty(tq.shape[:-1], device="cuda")
    status = torch.zeros(B * L * Hkv, dtype=torch.int32, device="cuda")

    def attend_step():
        kvc.kvc_i4_append(shape, rows, tk, tv, unit_status=status)
        kvc.kvc_i4_attn(shape, rows, tq, out, add_mass=True, row_lse=lse, workspace=aw)

    def evict_step():
        kvc.kvc_i4_evict(shape, rows, budget, 4, 32, unit_status=status, workspace=ew)

    calls = [attend_step, evict_step]
    if graph:
        keep = snapshot(rows)
        for f in calls:
            f()
        torch.cuda.synchronize()
        graphs = []
        for f in calls:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                f()
            graphs.append(gr)
        for t, t0 in zip(fields(rows), keep):
            t.copy_(t0)
        calls = [gr.replay for gr in graphs]
    for step in range(steps):
        for x in (tq, tk, tv):
            x.copy_(randn(g, *x.shape))
        mass0 = rows.mass.clone()
        n0 = rows.count.clone()
        calls[0]()
        torch.cuda.synchronize()
        at = n0.long()
        mass0.scatter_(1, at[:, None], 0.0)
        check_attention(c, tq, out, lse, mass0, add=True)
        calls[1]()
        torch.cuda.synchronize()
        assert int(status.abs().max()) == 0
        assert rows.count.tolist() == [budget] * 8
        assert rows.next_pos.tolist() == [301 + step] * 4 + [261 + step] * 4
        for u in range(8):
            p = rows.pos[u, :budget]
            assert len(set(p.tolist())) == budget
            assert set(range(4)) <= set(p.tolist())
            assert set(range(int(rows.next_pos[u]) - 32, int(rows.next_pos[u]))) <= set(p.tolist())


def test_calls_that_feed_each_other_without_a_pause(kvc):
    """Each call's outputs are the next one's inputs, and torch overwrites them right behind: the bits of the same calls
    with the device idle between them."""
    T, H, d = 200, 2, 128
    shape, g = kvc.make_shape(2, 1, H, H, d, T), gen(11)
    q0, k0, v0 = randn(g, 2, 1, H, T, d), randn(g, 2, 1, H, T, d), randn(g, 2, 1, H, T, d)
    space = lambda n: torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
    ws = space(kvc.kvc_prompt_attn_workspace_bytes(shape, T, True))
    docs = i32([[0] * 90 + [1] * 110] * 2)
    rows = kvc.I4Rows.allocate(shape, 2 * T)
    for t in fields(rows)[:6]:
        t.zero_()
    ws4, wse = space(kvc.kvc_i4_attn_workspace_bytes(shape, rows, T, True)), space(kvc.kvc_i4_evict_workspace_bytes(shape, rows, 150))

    def run(pause):
        torch.cuda.synchronize()
        rows.count.zero_(), rows.next_pos.zero_()
        a, b, c = torch.empty_like(q0), torch.empty_like(q0), torch.empty_like(q0)
        k_out, v_out = torch.zeros_like(k0), torch.zeros_like(v0)
        steps = [lambda: kvc.kvc_prompt_attn(shape, q0, k0, v0, a, workspace=ws),
                 lambda: kvc.kvc_prompt_attn(shape, a, k0, v0, b, docs=docs, workspace=ws),
                 lambda: a.zero_(),
                 lambda: kvc.kvc_prompt_attn(shape, b, b, v0, a, workspace=ws),
                 lambda: kvc.kvc_i4_append(shape, rows, a, b),
                 lambda: b.fill_(7.0),
                 lambda: kvc.kvc_i4_attn(shape, rows, a, c, add_mass=True, workspace=ws4),
                 lambda: kvc.kvc_i4_evict(shape, rows, 150, 4, 16, workspace=wse),
                 lambda: kvc.kvc_i4_append(shape, rows, c, a, n_new=i32([30, 50])),
                 lambda: kvc.kvc_i4_attn(shape, rows, c, a, workspace=ws4),
                 lambda: kvc.kvc_i4_read(shape, rows, k_out, v_out),
                 lambda: kvc.kvc_prompt_attn(shape, a, k_out, v_out, b, workspace=ws)]
        for s in steps:
            s()
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [t.clone() for t in (a, b, c, k_out, v_out, rows.mass[:, :180], rows.pos[:, :180], rows.count)]

    want = run(True)
    assert all(bool(torch.isfinite(t.float()).all()) for t in want)
    for _ in range(20):
        assert all(torch.equal(x, y) for x, y in zip(run(False), want))
