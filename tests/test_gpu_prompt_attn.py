"""kvc_prompt_attn against the 64-bit definition: lengths from none to long, odd sizes, head groups,
strides, masks that leave rows empty, documents, garbage where nothing is visible, other streams, graphs,
and the statistics it hands to kvc_score."""
import math

import pytest
import torch

from attn_reference import attend, close, visible

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


def tensor(g, B, L, H, n, d, layout):
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    if layout == "token":                                     # as a projection leaves it
        return r(B, L, n, H, d).transpose(2, 3)
    if layout == "padded":                                    # a view into larger rows and buffers
        return r(B, L, H, n + 3, d + 24)[:, :, :, 1:n + 1, 8:8 + d]
    return r(B, L, H, n, d)


class Case:
    def __init__(self, kvc, B=1, L=1, Hkv=2, G=4, d=128, n_q=1, T=1, q_len=None, kv_len=None, docs=None, softcap=0.0,
                 slopes=False, window=0, prefix=None, layout="head", seed=0, q_norm=2.0, scale=0.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.kvc, self.B, self.L, self.Hkv, self.G, self.d, self.n_q, self.T = kvc, B, L, Hkv, G, d, n_q, T
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        self.shape = kvc.make_shape(B, L, Hkv * G, Hkv, d, T)
        self.q = tensor(g, B, L, Hkv * G, n_q, d, layout)
        self.q.mul_(q_norm)
        self.k, self.v = tensor(g, B, L, Hkv, T, d, layout), tensor(g, B, L, Hkv, T, d, layout)
        self.out = tensor(g, B, L, Hkv * G, n_q, d, layout)
        self.out.fill_(7.0)
        self.lse = torch.full((B, L, Hkv * G, n_q), 7.0, device="cuda")
        self.q_len, self.kv_len = (None if x is None else i32(x) for x in (q_len, kv_len))
        self.docs = None if docs is None else i32(docs).expand(B, T).contiguous()
        self.slopes = torch.rand(Hkv * G, generator=g, device="cuda") * 0.05 if slopes else None
        self.softcap, self.window, self.scale = softcap, window, scale
        self.prefix = None if prefix is None else i32(prefix)
        self.status = torch.zeros(B * L * Hkv, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(max(1, kvc.kvc_prompt_attn_workspace_bytes(self.shape, n_q, docs is not None)),
                              dtype=torch.uint8, device="cuda")

    def run(self, stream=None, out=None, lse=None):
        mods = self.kvc.ScoreMods(self.softcap, self.slopes, self.window, self.prefix)
        self.kvc.kvc_prompt_attn(self.shape, self.q, self.k, self.v, self.out if out is None else out,
                                 q_len=self.q_len, kv_len=self.kv_len, docs=self.docs, mods=mods,
                                 softmax_scale=self.scale, row_lse=self.lse if lse is None else lse,
                                 unit_status=self.status, workspace=self.ws, stream=stream)

    def check(self):
        torch.cuda.synchronize()
        assert int(self.status.abs().max()) == 0
        scale = self.scale or 1 / math.sqrt(self.d)
        for b in range(self.B):
            nk = self.T if self.kv_len is None else max(0, min(self.T, int(self.kv_len[b])))
            nq = self.n_q if self.q_len is None else max(0, min(self.n_q, int(self.q_len[b])))
            p_q = torch.arange(nk - nq, nk, device="cuda")
            p_k = torch.arange(nk, device="cuda")
            pre = 0 if self.prefix is None else int(self.prefix[b])
            seen = visible(p_q, p_k, self.window, pre) & (p_q >= 0)[:, None]
            if self.docs is not None and nk:
                d = self.docs[b, :nk]
                seen = seen & (d[p_q.clamp(min=0)][:, None] == d[None, :]) & (d >= 0)[None, :]
            dist = (p_q[:, None] - p_k[None, :]).double()
            for l in range(self.L):
                for h in range(self.Hkv * self.G):
                    k, v = self.k[b, l, h // self.G, :nk].double(), self.v[b, l, h // self.G, :nk].double()
                    o, lse, _, e_o, e_l, _ = attend(self.q[b, l, h, :nq].double(), k, v, scale, seen, dist, self.softcap,
                                                    None if self.slopes is None else float(self.slopes[h]))
                    at = f"b{b} l{l} h{h}"
                    close(self.out[b, l, h, :nq], o, e_o, "out " + at)
                    close(self.lse[b, l, h, :nq], lse, e_l, "lse " + at)
            # rows behind the sequence's queries stay as they were
            assert bool((self.out[b, :, :, nq:] == 7).all()) and bool((self.lse[b, :, :, nq:] == 7).all())


CASES = {
    "one_key": dict(n_q=1, T=1),
    "one_key_d64": dict(n_q=1, T=1, d=64, G=1),
    "two": dict(n_q=2, T=2, B=2),
    "tile_edges": dict(n_q=128, T=128, G=1, Hkv=3),
    "past_tile": dict(n_q=129, T=257, G=1, layout="token"),
    "odd_group": dict(n_q=37, T=131, G=3, Hkv=2, d=64, layout="padded"),
    "five_heads": dict(n_q=70, T=70, G=5, Hkv=1, layout="token"),
    "seven_heads": dict(n_q=301, T=333, G=7, Hkv=1, d=64),
    "wide_group": dict(n_q=3, T=700, G=33, Hkv=1),
    "very_wide_group": dict(n_q=2, T=140, G=150, Hkv=1, d=64),
    "group_of_half_a_tile": dict(B=2, n_q=5, T=300, G=64, Hkv=2, q_len=[5, 2]),
    "group_of_a_tile": dict(n_q=3, T=300, G=128, Hkv=2, d=64),
    "layers": dict(B=2, L=3, n_q=65, T=200, G=2),
    "square": dict(n_q=600, T=600, G=4, Hkv=1),
    "chunk_of_long": dict(n_q=100, T=3001, G=4, Hkv=2),
    "decode": dict(B=3, n_q=1, T=5000, G=4, Hkv=2),
    "decode_long": dict(B=1, n_q=1, T=20011, G=8, Hkv=1, d=64),
    "draft": dict(B=2, n_q=6, T=2500, G=4, Hkv=2),
    "own_scale": dict(n_q=40, T=90, scale=0.3),
    "ragged": dict(B=5, n_q=90, T=300, q_len=[90, 1, 0, 17, 64], kv_len=[300, 1, 40, 17, 129]),
    "no_keys": dict(B=3, n_q=4, T=130, q_len=[4, 4, 2], kv_len=[0, 130, 0]),
    "more_queries_than_keys": dict(B=2, n_q=9, T=50, kv_len=[5, 50], prefix=[3, 0]),
    "lengths_out_of_range": dict(B=3, n_q=9, T=50, q_len=[-3, 400, 9], kv_len=[50, 4000, -7]),
    "softcap": dict(n_q=150, T=400, softcap=5.0, q_norm=8.0),
    "softcap_large": dict(n_q=33, T=100, softcap=50.0, d=64),
    "slopes": dict(n_q=150, T=400, slopes=True),
    "window_one": dict(n_q=200, T=300, window=1),
    "window": dict(n_q=300, T=900, window=77, G=2),
    "window_decode": dict(B=2, n_q=1, T=4000, window=100),
    "prefix": dict(B=3, n_q=200, T=260, prefix=[0, 100, 260]),
    "prefix_window": dict(B=2, n_q=200, T=600, prefix=[130, 300], window=20),
    "bidirectional": dict(n_q=190, T=190, prefix=[190], slopes=True),
    "docs": dict(n_q=700, T=700, G=2, docs=[0] * 100 + [1] * 1 + [2] * 399 + [5] * 200),
    "docs_padding": dict(n_q=300, T=300, docs=[0] * 130 + [-1] * 40 + [3] * 100 + [-1] * 30),
    "docs_mixed_order": dict(n_q=260, T=400, docs=[i % 3 for i in range(400)], window=50),
    "docs_tail": dict(n_q=5, T=1000, docs=[0] * 990 + [1] * 10),
    "everything": dict(B=3, L=2, G=3, n_q=140, T=500, d=64, q_len=[140, 50, 3], kv_len=[500, 222, 3], softcap=10.0,
                       slopes=True, window=60, prefix=[30, 0, 2], docs=[0] * 250 + [1] * 250, layout="token"),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_the_definition(kvc, name):
    c = Case(kvc, **CASES[name])
    c.run()
    c.check()


@pytest.mark.parametrize("n_q", [1, 5, 150])
def test_rows_that_nothing_sees_may_hold_any_bits(kvc, n_q):
    """NaN behind kv_len, at tokens of negative documents, and before the window of every query."""
    c = Case(kvc, B=2, n_q=n_q, T=700, G=2, kv_len=[333, 700], docs=[0] * 40 + [-1] * 60 + [0] * 600, window=150)
    for x in (c.k, c.v):
        x[0, :, :, 333:] = float("nan")
        x[:, :, :, 40:100] = float("inf")
        x[0, :, :, :max(0, 333 - n_q - 149)] = float("nan")
        x[1, :, :, :max(0, 700 - n_q - 149)] = float("nan")
    c.run()
    c.check()


def test_documents_that_no_query_has_may_hold_any_bits(kvc):
    """A chunk of the second document: the first one's rows, some in the same key tile, are NaN."""
    c = Case(kvc, n_q=150, T=700, G=2, docs=[0] * 430 + [1] * 270)
    for x in (c.k, c.v):
        x[:, :, :, :430] = float("nan")
    c.run()
    c.check()


@pytest.mark.parametrize("kw", [dict(window=200), dict(window=5000), dict(window=300, prefix=[700, 0])])
def test_window_over_a_long_cache(kvc, kw):
    """Splits of the keys follow the window where nothing else is seen."""
    c = Case(kvc, B=2, n_q=2, T=30000, Hkv=1, G=4, d=64, kv_len=[30000, 17001], **kw)
    c.run()
    c.check()


def test_two_streams_at_once(kvc):
    """Two calls that overlap, each with its own workspace."""
    cases = [Case(kvc, B=2, n_q=1, T=20000, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_large_logits_stay_finite(kvc):
    c = Case(kvc, n_q=140, T=300, q_norm=60.0, seed=3)
    c.run()
    c.check()


def test_logits_that_grow_along_the_keys(kvc):
    """The running maximum rises in every tile, by a lot and by a little."""
    c = Case(kvc, n_q=64, T=1500, Hkv=1, G=2, prefix=[1500], seed=5)
    ramp = torch.linspace(0.05, 6.0, 1500, device="cuda")[:, None]
    q = torch.randn(128, device="cuda")
    c.q[:] = q.to(torch.bfloat16)
    c.k[0, 0, 0] = (ramp * q / q.norm()).to(torch.bfloat16)
    c.run()
    c.check()


def test_long_cache_past_32_bit_offsets(kvc):
    """Keys of the last units start past 2^31 elements."""
    B, T, d = 5, 1 << 22, 128
    k = torch.empty(B, 1, 1, T, d, dtype=torch.bfloat16, device="cuda")
    c = Case(kvc, B=B, Hkv=1, G=2, n_q=1, T=1, d=d)
    c.shape, c.T = kvc.make_shape(B, 1, 2, 1, d, T), T
    c.k, c.v = k, torch.empty_like(k)
    for x in (c.k, c.v):
        x[:, :, :, -600:] = torch.randn(B, 1, 1, 600, d, device="cuda").to(torch.bfloat16)
    c.window = 500
    c.ws = torch.empty(max(1, kvc.kvc_prompt_attn_workspace_bytes(c.shape, 1, False)), dtype=torch.uint8, device="cuda")
    full = c.k, c.v
    c.run()
    torch.cuda.synchronize()
    # the same through the last rows alone
    s = Case(kvc, B=B, Hkv=1, G=2, n_q=1, T=600, d=d)
    s.q, s.k, s.v, s.window, s.out, s.lse = c.q, full[0][:, :, :, -600:], full[1][:, :, :, -600:], 500, c.out, c.lse
    s.check()


def test_same_bits_twice_and_on_another_stream(kvc):
    for kw in (dict(n_q=500, T=900, B=2), dict(n_q=1, T=9000, B=2)):
        c = Case(kvc, **kw)
        c.run()
        torch.cuda.synchronize()
        first, lse = c.out.clone(), c.lse.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        c.out.zero_()
        s.wait_stream(torch.cuda.current_stream())
        c.run(stream=s)
        s.synchronize()
        assert torch.equal(first, c.out) and torch.equal(lse, c.lse)


@pytest.mark.parametrize("kw", [dict(n_q=300, T=700, docs=[0] * 300 + [1] * 400), dict(n_q=1, T=9000)])
def test_replayed_from_a_graph_with_new_lengths(kvc, kw):
    """Lengths are read on the device, so a replay follows what they hold then."""
    c = Case(kvc, B=2, kv_len=[kw["T"], 40], **kw)
    c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    c.kv_len.copy_(torch.tensor([kw["T"] - 130, kw["T"]], dtype=torch.int32))
    c.out.fill_(7.0)
    g.replay()
    c.check()


def test_two_graphs_share_a_workspace(kvc):
    a, b = Case(kvc, B=2, n_q=1, T=9000), Case(kvc, B=2, n_q=1, T=7000, seed=1)
    b.ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    a.ws = b.ws
    graphs = []
    for c in (a, b):
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    a.check()
    b.check()


def test_row_statistics_feed_the_window_score(kvc):
    """row_lse of the last queries gives kvc_score the statistics that it would compute itself."""
    B, Hkv, G, d, T, W = 1, 2, 4, 128, 2000, 32
    c = Case(kvc, B=B, Hkv=Hkv, G=G, d=d, n_q=W, T=T)
    c.run()
    scores = []
    ws = torch.empty(kvc.kvc_score_workspace_bytes(c.shape, W), dtype=torch.uint8, device="cuda")
    for lse in (None, c.lse):
        s = torch.empty(B * Hkv, T, device="cuda")
        kvc.kvc_score(c.shape, c.k, c.q, W, 0.0, None, 1, 0, s, None, None, ws, row_lse=lse)
        torch.cuda.synchronize()
        scores.append(s.double())
    # each side's row statistics are off by at most (d + 4) u of the largest sum |q||k| * scale of a row,
    # which moves a weight, and so a sum of weights, by that relative amount
    big = float((c.q.double().abs().view(B, Hkv, G * W, d) @ c.k.double().abs().view(B, Hkv, T, d).transpose(2, 3)).max())
    bound = 2 * (2 * (d + 4) * 2.0 ** -24 * big / math.sqrt(d) + 2.0 ** -21 + T * 2.0 ** -24)
    assert float(((scores[0] - scores[1]).abs() / scores[0]).max()) < bound


def test_workspace_too_small_is_refused(kvc):
    c = Case(kvc, B=1, Hkv=1, G=1, n_q=1, T=50000)
    need = kvc.kvc_prompt_attn_workspace_bytes(c.shape, 1, False)
    if need == 0:
        pytest.skip("no workspace at this size")
    c.ws = torch.empty(need - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(kvc.KvcError) as e:
        c.run()
    assert e.value.code == 3


@pytest.mark.parametrize("empty", ["no_keys", "padding"])
@pytest.mark.parametrize("G, n_q", [(4, 32), (4, 150), (3, 42), (3, 150)])
@pytest.mark.parametrize("d", [64, 128])
def test_blocks_of_queries_that_walk_no_key(kvc, d, G, n_q, empty):
    """Every query of many blocks (one or two row tiles, queries by tensor copies or by plain loads) sees nothing: the
    outputs, staged where the queries land, are zeros whenever the queries land."""
    B, T = 100, 300
    c = Case(kvc, B=B, Hkv=2, G=G, d=d, n_q=n_q, T=T, q_norm=500.0, **(
        dict(kv_len=[0] * B) if empty == "no_keys" else dict(docs=[0] * (T - n_q) + [-1] * n_q)))
    for _ in range(20):
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        c.run()
        torch.cuda.synchronize()
        assert int(c.status.abs().max()) == 0
        assert int((c.out != 0).sum()) == 0 and bool((c.lse == -math.inf).all())
