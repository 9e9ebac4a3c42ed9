"""Cases of the prompt attention and of the 4-bit cache: what they compute, in plain
torch operations, and the calls that a user's program makes of the library.

Operators (each `op` of a case is one pass of a program):
  prompt  kvc_prompt_attn: attention of a prompt chunk or of single tokens over bf16
          keys and values, with a tanh cap, a distance bias, a sliding window,
          documents and a prefix; outputs and row log-sum-exps
  store   kvc_i4_append + kvc_i4_read: rows quantised into a 4-bit cache, and read back
  attn    kvc_i4_attn: attention over the 4-bit cache, softmax weights added to its mass
  evict   kvc_i4_append + kvc_i4_evict + kvc_i4_read: new rows in, the rows with the
          least mass out, and the rows that remain
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
G32, ROW = 0, 1                       # a bf16 scale per 32 elements, or an fp16 scale per row


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one layer of a first request's prompt, where launches and latency count
        _prompt("prompt_short", batch=1, heads=32, kv=8, d=128, n_q=300, n_k=300),
        # one layer of a long prompt, causal
        _prompt("prompt_causal_8k", batch=1, heads=32, kv=8, d=128, n_q=8192, n_k=8192),
        # documents packed into one sequence, capped scores
        _prompt("prompt_docs_capped", batch=1, heads=16, kv=4, d=128, n_q=8000, n_k=8000, softcap=30.0, docs=9,
                layout="token"),
        # a padded batch with a bidirectional prefix, distance bias and odd head groups
        _prompt("prompt_prefix_bias", batch=4, heads=12, kv=4, d=64, n_q=1901, n_k=2333, slopes=True, prefix=257,
                ragged=True, layout="token"),
        # one decode step of a batch over bf16 caches, sliding window off, capped scores
        _prompt("prompt_decode_32k", batch=16, heads=32, kv=8, d=128, n_q=1, n_k=32768, softcap=50.0, ragged=True),
        # the rows of one new token, every layer
        _store("store_token", batch=1, layers=36, kv=8, d=128, n=1, mode=G32),
        # a long prompt's rows, ragged batch
        _store("store_prompt", batch=3, layers=4, kv=8, d=128, n=30011, mode=G32, ragged=True),
        # one decode step of one layer over a budgeted cache
        _attn("attn_2k", batch=1, layers=1, heads=32, kv=8, d=128, n_q=1, cap=2304, lo=2048, mode=G32, mass=True),
        # long caches of a batch
        _attn("attn_128k", batch=4, layers=1, heads=32, kv=8, d=128, n_q=1, cap=131072, lo=100000, mode=G32, mass=True),
        # drafted tokens of a batch checked at once, ragged, row scales, capped and windowed
        _attn("attn_draft", batch=8, layers=1, heads=24, kv=8, d=64, n_q=5, cap=9001, lo=300, mode=ROW, softcap=30.0,
              slopes=True, window=4096, mass=False),
        # one token in, one row out, one layer
        _evict("evict_step", batch=1, layers=1, kv=8, d=128, n=1, budget=2048, mode=G32),
        # a chunk in, as many rows out, every layer
        _evict("evict_chunk", batch=1, layers=36, kv=8, d=128, n=100, budget=2048, mode=ROW),
    ]


def _prompt(name, **kw):
    c = dict(op="prompt", batch=1, heads=32, kv=8, d=128, n_q=1, n_k=1, softcap=0.0, slopes=False, window=0, docs=0,
             prefix=0, ragged=False, layout="head")
    return dict(c, **kw, **({"name": name} if name else {}))


def _store(name, **kw):
    c = dict(op="store", batch=1, layers=1, kv=8, d=128, n=1, mode=G32, ragged=False)
    return dict(c, **kw, **({"name": name} if name else {}))


def _attn(name, **kw):
    c = dict(op="attn", batch=1, layers=1, heads=32, kv=8, d=128, n_q=1, cap=256, lo=1, mode=G32, softcap=0.0,
             slopes=False, window=0, mass=False)
    return dict(c, **kw, **({"name": name} if name else {}))


def _evict(name, **kw):
    c = dict(op="evict", batch=1, layers=1, kv=8, d=128, n=1, budget=64, mode=G32)
    return dict(c, **kw, **({"name": name} if name else {}))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "store", "attn", "attn", "evict"])
    d, kv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    mode = rng.choice([G32, ROW])
    if op == "prompt":
        group = rng.choice([1, 2, 3, 4, 5, 7, 8])
        n_k = _log(rng, 1, 32768)
        n_q = n_k if rng.random() < 0.5 else _log(rng, 1, n_k)
        while n_q * n_k * kv * group > 32 * 8192 * 8192:
            n_q = max(1, n_q // 2)
        batch = max(1, min(16, (1 << 31) // max(1, n_q * n_k * kv * group), _log(rng, 1, 16),
                           (1 << 29) // (n_k * kv * d)))
        return _prompt(None, batch=batch, heads=kv * group, kv=kv, d=d, n_q=n_q, n_k=n_k,
                       softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), slopes=rng.random() < 0.3,
                       window=rng.choice([0, 0, _log(rng, 1, 8192)]), docs=rng.choice([0, 0, rng.randint(2, 20)]),
                       prefix=rng.choice([0, 0, _log(rng, 1, n_k)]), ragged=rng.random() < 0.5,
                       layout=rng.choice(["head", "token"]))
    if op == "store":
        layers, n = _log(rng, 1, 36), _log(rng, 1, 30011)
        return _store(None, batch=max(1, min(4, 360000 * 8 // (n * layers * kv))), layers=layers, kv=kv, d=d,
                      n=min(n, 360000 * 8 // (layers * kv)), mode=mode,
                      ragged=rng.random() < 0.5)
    if op == "attn":
        group, n_q = rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([1, 1, 1, 2, 3, 5, 17])
        cap = _log(rng, 1, 131072)
        units = max(1, min(64, (1 << 22) // (cap * group * n_q // 4 + 1)))
        return _attn(None, batch=max(1, min(8, units // kv)), layers=1, heads=kv * group, kv=kv, d=d, n_q=n_q, cap=cap,
                     lo=rng.randint(0, cap), mode=mode, softcap=rng.choice([0.0, 0.0, 30.0]),
                     slopes=rng.random() < 0.3, window=rng.choice([0, 0, _log(rng, 1, 65536)]),
                     mass=rng.random() < 0.6)
    budget = _log(rng, 160, 16384)
    layers = max(1, min(36, (288 * 2048) // (budget * kv)))
    return _evict(None, batch=1, layers=rng.randint(1, layers), kv=kv, d=d, n=_log(rng, 1, 128), budget=budget, mode=mode)


# ------------------------------------------------------------------------------ shapes a case fixes

def _units(c):
    return c["batch"] * c.get("layers", 1) * c["kv"]


def _lens(c):
    """(q_len, kv_len) of each sequence of a prompt case: whole, or ragged with one full sequence."""
    q, k = [c["n_q"]] * c["batch"], [c["n_k"]] * c["batch"]
    if c["ragged"]:
        r = np.random.RandomState(c["n_k"] * 7 + c["n_q"])
        k = [c["n_k"]] + [int(r.randint(1, c["n_k"] + 1)) for _ in range(c["batch"] - 1)]
        q = [min(c["n_q"], n) if i % 3 == 0 else int(r.randint(1, min(c["n_q"], n) + 1)) for i, n in enumerate(k)]
    return q, k


def _doc_ids(c):
    """Document of each token, [batch, n_k]: runs of unequal length."""
    r = np.random.RandomState(c["n_k"] * 3 + c["docs"])
    out = np.zeros((c["batch"], c["n_k"]), np.int32)
    for b in range(c["batch"]):
        out[b, r.randint(0, c["n_k"], c["docs"] - 1)] = 1
    return np.cumsum(out, axis=1).astype(np.int32)


def _counts(c):
    """Rows in use of each sequence's units of an attn case; the first is full."""
    r = np.random.RandomState(c["cap"] * 5 + c["lo"])
    return [c["cap"]] + [int(r.randint(c["lo"], c["cap"] + 1)) for _ in range(c["batch"] - 1)]


def _new(c):
    """Rows that each sequence of a store case appends: n, or ragged with one full sequence."""
    r = np.random.RandomState(c["n"] * 11)
    return [c["n"] if i == 0 or not c["ragged"] else int(r.randint(0, c["n"] + 1)) for i in range(c["batch"])]


def _row_bytes(c):
    return 2 * (c["d"] // 2 + (2 * (c["d"] // 32) if c["mode"] == G32 else 2))


def work(case):
    c = case
    if c["op"] == "prompt":
        q, k = _lens(c)
        pairs = 0
        ids = _doc_ids(c) if c["docs"] else None
        for b in range(c["batch"]):
            p = np.arange(k[b] - q[b], k[b], dtype=np.int64)
            first, last = np.zeros_like(p), np.full_like(p, k[b])
            if c["docs"]:
                first = np.searchsorted(ids[b, :k[b]], ids[b, p], "left")
                last = np.searchsorted(ids[b, :k[b]], ids[b, p], "right")
            lo = np.maximum(first, p - c["window"] + 1) if c["window"] else first
            pre = np.minimum(last, c["prefix"])
            pairs += int((np.maximum(pre - first, 0) + np.maximum(p + 1 - np.maximum(lo, pre), 0)).sum())
        rows = sum(q) * c["heads"]
        return {"bytes": rows * (4 * c["d"] + 4) + sum(k) * c["kv"] * 4 * c["d"], "flops": 4 * c["d"] * c["heads"] * pairs}
    u = _units(c)
    if c["op"] == "store":
        return {"bytes": sum(_new(c)) * c["layers"] * c["kv"] * (8 * c["d"] + 2 * _row_bytes(c)), "flops": 0}
    if c["op"] == "attn":
        keys = sum(min(n, c["window"] + c["n_q"]) if c["window"] else n for n in _counts(c)) * c["kv"] * c["layers"]
        rows = c["batch"] * c["layers"] * c["heads"] * c["n_q"]
        return {"bytes": keys * (_row_bytes(c) + 4 + (8 if c["mass"] else 0)) + rows * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * keys * (c["heads"] // c["kv"]) * c["n_q"]}
    return {"bytes": u * (c["budget"] * (_row_bytes(c) + 4 * c["d"] + 8) + c["n"] * (4 * c["d"] + 3 * _row_bytes(c))),
            "flops": 0}


# ------------------------------------------------------------------------------ inputs

Q_NORM = 2.0                          # logits of about 2 standard deviations: rows attend to few of many keys


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def _tensor(g, c, heads, n):
    """A [B][1][H][n][d] tensor, stored head by head or token by token as a projection leaves it."""
    if c["layout"] == "token":
        return _randn(g, c["batch"], 1, n, heads, c["d"]).transpose(2, 3)
    return _randn(g, c["batch"], 1, heads, n, c["d"])


def _slopes(heads):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], device=DEV)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Rows:
    """The arrays of a 4-bit cache: codes, scales, positions, accumulated weight, rows in use."""

    def __init__(self, units, cap, d, mode):
        e = lambda *s, dt: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
        ns, sdt = (d // 32, torch.bfloat16) if mode == G32 else (1, torch.float16)
        self.mode, self.d, self.cap = mode, d, cap
        self.k, self.v = e(units, cap, d // 2, dt=torch.uint8), e(units, cap, d // 2, dt=torch.uint8)
        self.k_scale, self.v_scale = e(units, cap, ns, dt=sdt), e(units, cap, ns, dt=sdt)
        self.pos, self.mass = e(units, cap, dt=torch.int32), e(units, cap, dt=torch.float32)
        self.counters = e(2, units, dt=torch.int32)          # rows in use, next position
        self.count, self.next_pos = self.counters[0], self.counters[1]


def _fill(rows, g, counts):
    """Rows that a cache holds after a while: quantised normal vectors, positions with gaps, past weights."""
    u, cap = rows.pos.shape
    for codes, scale in ((rows.k, rows.k_scale), (rows.v, rows.v_scale)):
        step = max(1, (1 << 27) // (cap * rows.d))
        for a in range(0, u, step):
            x = torch.randn((min(step, u - a), cap, rows.d), generator=g, device=DEV)
            codes[a:a + step], scale[a:a + step] = _quantise(x.to(torch.bfloat16), rows.mode)
    gap = torch.randint(1, 4, (u, cap), generator=g, device=DEV)
    rows.pos.copy_(torch.cumsum(gap, 1) - gap[:, :1])
    rows.mass.copy_(torch.rand((u, cap), generator=g, device=DEV) * 4)
    rows.count.copy_(counts)
    last = rows.pos.gather(1, (counts.long() - 1).clamp(min=0)[:, None])[:, 0]
    rows.next_pos.copy_(torch.where(counts > 0, last + 1, torch.zeros_like(last)))


def _shape(c, n):
    import budgeted_kv_cache_gb300 as kvc
    return kvc.make_shape(c["batch"], c.get("layers", 1), c.get("heads", c["kv"]), c["kv"], c["d"], n)


def prepare(case, seed):
    c, g, s = dict(case), _gen(seed), {"case": dict(case)}
    if c["op"] == "prompt":
        q_len, kv_len = _lens(c)
        s["q"] = _tensor(g, c, c["heads"], c["n_q"]) * Q_NORM
        s["k"], s["v"] = _tensor(g, c, c["kv"], c["n_k"]), _tensor(g, c, c["kv"], c["n_k"])
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(c["batch"], 1, c["heads"], c["n_q"], device=DEV)
        s["q_len"], s["kv_len"] = (_int(q_len), _int(kv_len)) if c["ragged"] else (None, None)
        s["docs"] = torch.from_numpy(_doc_ids(c)).to(DEV) if c["docs"] else None
        s["slopes"] = _slopes(c["heads"]) if c["slopes"] else None
        s["prefix"] = _int([c["prefix"]] * c["batch"]) if c["prefix"] else None
        if own:
            import budgeted_kv_cache_gb300 as kvc
            s["shape"] = _shape(c, c["n_k"])
            s["mods"] = kvc.ScoreMods(c["softcap"], s["slopes"], c["window"], s["prefix"])
            s["ws"] = _workspace(kvc.kvc_prompt_attn_workspace_bytes(s["shape"], c["n_q"], s["docs"] is not None))
        return s
    u, d = _units(c), c["d"]
    cap = {"store": c.get("n"), "attn": c.get("cap"), "evict": c.get("budget", 0) + c.get("n", 0)}[c["op"]]
    rows = s["rows"] = Rows(u, cap, d, c["mode"])
    per_seq = lambda v: _int(v).repeat_interleave(u // c["batch"])  # noqa: E731
    if c["op"] == "attn":
        _fill(rows, g, per_seq(_counts(c)))
        s["q"] = _randn(g, c["batch"], c["layers"], c["heads"], c["n_q"], d) * Q_NORM
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(s["q"].shape[:-1], device=DEV)
        s["slopes"] = _slopes(c["heads"]) if c["slopes"] else None
    else:
        if c["op"] == "evict":
            _fill(rows, g, _int([c["budget"]] * u))
        n = c["n"]
        s["k"], s["v"] = _randn(g, c["batch"], c["layers"], c["kv"], n, d), _randn(g, c["batch"], c["layers"], c["kv"], n, d)
        s["k_out"] = torch.zeros(c["batch"], c["layers"], c["kv"], n if c["op"] == "store" else c["budget"], d,
                                 dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.zeros_like(s["k_out"])
        s["empty"] = torch.zeros_like(rows.counters)
        s["n_new"] = _int(_new(c)) if c.get("ragged") else None
    if own:
        import budgeted_kv_cache_gb300 as kvc
        s["shape"] = _shape(c, cap)
        s["cache"] = kvc.I4Rows(rows.k, rows.v, rows.k_scale, rows.v_scale, rows.pos, rows.count, rows.next_pos,
                                rows.mass, c["mode"])
        if c["op"] == "attn":
            s["mods"] = kvc.ScoreMods(c["softcap"], s["slopes"], c["window"])
            s["ws"] = _workspace(kvc.kvc_i4_attn_workspace_bytes(s["shape"], s["cache"], c["n_q"], c["mass"]))
        if c["op"] == "evict":
            s["ws"] = _workspace(kvc.kvc_i4_evict_workspace_bytes(s["shape"], s["cache"], c["budget"]))
    return s


def _workspace(n):
    return torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------------------ plain forms

def _quantise(x, mode):
    """Codes (two to a byte, the even element in the low half) and scales of bf16 rows."""
    d = x.shape[-1]
    f = x.float().unflatten(-1, (d // 32, 32) if mode == G32 else (1, d))
    a = f.abs().amax(-1)
    scale = (a / 7).to(torch.bfloat16 if mode == G32 else torch.float16).float()
    scale = torch.where(a > 0, scale.clamp(min=2.0 ** (-133 if mode == G32 else -24)), torch.ones_like(scale))
    code = torch.round(f / scale[..., None]).clamp(-7, 7).flatten(-2).to(torch.int32)
    return ((code[..., 0::2] & 15) | ((code[..., 1::2] & 15) << 4)).to(torch.uint8), \
        scale.to(torch.bfloat16 if mode == G32 else torch.float16)


def _values(codes, scale, d):
    """fp32 values that codes and scales stand for."""
    x = codes.to(torch.int32)
    x = torch.stack((x & 15, x >> 4), -1).flatten(-2)
    x = ((x ^ 8) - 8).float()
    return (x.unflatten(-1, (scale.shape[-1], -1)) * scale.float()[..., None]).flatten(-2)


def _attend(c, q, k, v, slopes, dist, visible):
    """Softmax weights, outputs and row log-sum-exps of q [B,L,heads,n_q,d] over k, v [B,L,kv,T,d]; `visible` and `dist`
    (p_q - p_k) are [B,L or 1,kv or 1,1,n_q,T].  A row that sees nothing has output 0 and -inf."""
    g = c["heads"] // c["kv"]
    rows = q.float().unflatten(2, (c["kv"], g)).flatten(3, 4)
    x = (rows @ k.transpose(-1, -2)).unflatten(3, (g, c["n_q"])) * (1 / math.sqrt(c["d"]))
    if c["softcap"] > 0:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    if slopes is not None:
        x = x - slopes.view(1, 1, c["kv"], g, 1, 1) * dist.abs()
    x = torch.where(visible, x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    out = (p.flatten(3, 4) @ v).unflatten(3, (g, c["n_q"])).flatten(2, 3)
    lse = torch.where(total > 0, m + torch.log(total), float("-inf")).flatten(2, 3)[..., 0]
    return p, out, lse


def _prompt_visible(c, s):
    """visible [B,1,1,1,n_q,n_k] and distances p_q - p_k of a prompt case."""
    i, j = torch.arange(c["n_q"], device=DEV), torch.arange(c["n_k"], device=DEV)
    q_len = s["q_len"] if s["q_len"] is not None else torch.full((c["batch"],), c["n_q"], device=DEV)
    kv_len = s["kv_len"] if s["kv_len"] is not None else torch.full((c["batch"],), c["n_k"], device=DEV)
    p = (kv_len - q_len).view(-1, 1, 1) + i.view(1, -1, 1)
    dist = p - j
    ok = dist >= 0
    if c["window"]:
        ok = ok & (dist < c["window"])
    if s["prefix"] is not None:
        ok = ok | (j < s["prefix"].view(-1, 1, 1))
    if s["docs"] is not None:
        own_doc = s["docs"].long().gather(1, p[:, :, 0].clamp(0, c["n_k"] - 1).long())
        ok = ok & (own_doc[:, :, None] == s["docs"][:, None, :])
    ok = ok & (j < kv_len.view(-1, 1, 1))
    live = i.view(1, -1) < q_len.view(-1, 1)
    return ok[:, None, None, None], dist[:, None, None, None], live[:, None, None]


def _plain_prompt(c, s):
    visible, dist, live = _prompt_visible(c, s)
    _, out, lse = _attend(c, s["q"], s["k"].float(), s["v"].float(), s["slopes"], dist, visible)
    s["out"].copy_(torch.where(live[..., None], out, s["out"]))
    s["lse"].copy_(torch.where(live, lse, s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_append(c, s):
    """New rows behind those in use, n_new of each sequence."""
    r, u, n = s["rows"], _units(c), c["n"]
    i = torch.arange(n, device=DEV)
    slot = r.count[:, None] + i
    n_new = torch.full((c["batch"],), n, device=DEV) if s["n_new"] is None else s["n_new"]
    n_new = n_new.repeat_interleave(u // c["batch"])[:, None]
    live = i < n_new
    at = lambda i, x: i.view(u, n, *[1] * (x.dim() - 2)).expand_as(x)  # noqa: E731
    put = lambda x, new: x.scatter_(1, at(slot, new), torch.where(at(live, new), new, x.gather(1, at(slot, new))))  # noqa: E731
    for x, codes, scale in ((s["k"], r.k, r.k_scale), (s["v"], r.v, r.v_scale)):
        q, sc = _quantise(x.reshape(u, n, c["d"]), c["mode"])
        put(codes, q)
        put(scale, sc)
    put(r.pos, r.next_pos[:, None] + i.int())
    put(r.mass, torch.zeros(u, n, device=DEV))
    r.counters.add_(n_new.int()[:, 0])


def _plain_read(c, s):
    r, n = s["rows"], s["k_out"].shape[3]
    used = (torch.arange(n, device=DEV) < r.count[:, None])[..., None]
    for codes, scale, out in ((r.k, r.k_scale, s["k_out"]), (r.v, r.v_scale, s["v_out"])):
        x = _values(codes[:, :n], scale[:, :n], c["d"]).to(torch.bfloat16)
        out.copy_(torch.where(used, x, out.view(x.shape)).view(out.shape))


def _plain_store(c, s):
    s["rows"].counters.copy_(s["empty"])
    _plain_append(c, s)
    _plain_read(c, s)
    return {"k": s["k_out"], "v": s["v_out"], "pos": s["rows"].pos, "counters": s["rows"].counters}


def _attn_visible(c, r):
    slot = torch.arange(r.cap, device=DEV)
    p = (r.next_pos - c["n_q"])[:, None] + torch.arange(c["n_q"], device=DEV)
    dist = p[:, :, None] - r.pos[:, None, :]
    ok = (dist >= 0) & (slot < r.count[:, None])[:, None, :]
    if c["window"]:
        ok = ok & (dist < c["window"])
    shape = (c["batch"], c["layers"], c["kv"], 1, c["n_q"], r.cap)
    return ok.view(shape), dist.view(shape)


def _plain_attn(c, s):
    r = s["rows"]
    visible, dist = _attn_visible(c, r)
    lead = (c["batch"], c["layers"], c["kv"])
    k, v = (_values(a, b, c["d"]).view(*lead, r.cap, c["d"]) for a, b in ((r.k, r.k_scale), (r.v, r.v_scale)))
    p, out, lse = _attend(c, s["q"], k, v, s["slopes"], dist, visible)
    s["out"].copy_(out)
    s["lse"].copy_(lse)
    if c["mass"]:
        r.mass.add_(p.sum((3, 4)).view(r.mass.shape))
    return {"out": s["out"], "lse": s["lse"], "mass": r.mass}


N_SINK, N_RECENT = 4, 128


def _plain_evict(c, s):
    _plain_append(c, s)
    r, cap, budget = s["rows"], s["rows"].cap, c["budget"]
    slot = torch.arange(cap, device=DEV)
    used = slot < r.count[:, None]
    kept = (r.pos < N_SINK) | (r.pos >= (r.next_pos - N_RECENT)[:, None])
    out = used & ~kept
    # least mass first, of equal mass the later position first
    first = torch.argsort(r.pos, dim=1, descending=True, stable=True)
    mass = torch.where(out, r.mass, float("inf")).gather(1, first)
    order = first.gather(1, torch.argsort(mass, dim=1, stable=True))
    rank = torch.empty_like(order).scatter_(1, order, slot.expand_as(order))
    over = (r.count - budget).clamp(min=0)[:, None]
    victim = out & (rank < over)
    # holes below the budget, in order, take the kept rows behind it, in order
    hole, donor = victim & (slot < budget), used & ~victim & (slot >= budget)
    donors = torch.where(donor, slot, cap).sort(1).values
    src = torch.where(hole, donors.gather(1, (torch.cumsum(hole, 1) - 1).clamp(min=0)), slot.expand_as(order)).clamp(max=cap - 1)
    for x in (r.k, r.v, r.k_scale, r.v_scale):
        x.copy_(x.gather(1, src[..., None].expand_as(x)))
    r.pos.copy_(r.pos.gather(1, src))
    r.mass.copy_(r.mass.gather(1, src))
    r.count.copy_(torch.minimum(r.count, torch.full_like(r.count, budget)))
    _plain_read(c, s)
    return {"k": s["k_out"], "v": s["v_out"], "pos": r.pos, "mass": r.mass, "counters": r.counters}


# ------------------------------------------------------------------------------ the library's calls

def _own_prompt(c, s):
    import budgeted_kv_cache_gb300 as kvc
    kvc.kvc_prompt_attn(s["shape"], s["q"], s["k"], s["v"], s["out"], q_len=s["q_len"], kv_len=s["kv_len"],
                        docs=s["docs"], mods=s["mods"], row_lse=s["lse"], workspace=s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_store(c, s):
    import budgeted_kv_cache_gb300 as kvc
    s["rows"].counters.copy_(s["empty"])
    kvc.kvc_i4_append(s["shape"], s["cache"], s["k"], s["v"], n_new=s["n_new"])
    kvc.kvc_i4_read(s["shape"], s["cache"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"], "pos": s["rows"].pos, "counters": s["rows"].counters}


def _own_attn(c, s):
    import budgeted_kv_cache_gb300 as kvc
    kvc.kvc_i4_attn(s["shape"], s["cache"], s["q"], s["out"], mods=s["mods"], add_mass=c["mass"], row_lse=s["lse"],
                    workspace=s["ws"])
    return {"out": s["out"], "lse": s["lse"], "mass": s["rows"].mass}


def _own_evict(c, s):
    import budgeted_kv_cache_gb300 as kvc
    kvc.kvc_i4_append(s["shape"], s["cache"], s["k"], s["v"], n_new=s["n_new"])
    kvc.kvc_i4_evict(s["shape"], s["cache"], c["budget"], N_SINK, N_RECENT, workspace=s["ws"])
    kvc.kvc_i4_read(s["shape"], s["cache"], s["k_out"], s["v_out"])
    r = s["rows"]
    return {"k": s["k_out"], "v": s["v_out"], "pos": r.pos, "mass": r.mass, "counters": r.counters}


def run(state):
    c = state["case"]
    if own:
        return {"prompt": _own_prompt, "store": _own_store, "attn": _own_attn, "evict": _own_evict}[c["op"]](c, state)
    return {"prompt": _plain_prompt, "store": _plain_store, "attn": _plain_attn, "evict": _plain_evict}[c["op"]](c, state)


# ------------------------------------------------------------------------------ the definitions in 64 bits

def _row64(x, k, v, capped, minus, seen):
    """One head's rows: out, lse and weights from logits x in 64 bits."""
    if capped > 0:
        x = torch.tanh(x / capped) * capped
    if minus is not None:
        x = x - minus
    x = x.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - lse.masked_fill(torch.isinf(lse), 0.0)[:, None])
    return w @ v, lse, w


def _exact_prompt(c, s):
    q_len, kv_len = _lens(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    g = c["heads"] // c["kv"]
    ids = torch.from_numpy(_doc_ids(c)).to(DEV) if c["docs"] else None
    step = max(1, (1 << 26) // c["n_k"])
    for b in range(c["batch"]):
        nk, nq = kv_len[b], q_len[b]
        j = torch.arange(nk, device=DEV)
        for h in range(c["heads"]):
            k, v = s["k"][b, 0, h // g, :nk].double(), s["v"][b, 0, h // g, :nk].double()
            for a in range(0, nq, step):
                e = min(nq, a + step)
                p = torch.arange(nk - nq + a, nk - nq + e, device=DEV)[:, None]
                far = (p - j).double()
                seen = (far >= 0) & ((far < c["window"]) if c["window"] else True)
                seen = seen | (j < c["prefix"])
                if ids is not None:
                    seen = seen & (ids[b, :nk][p] == ids[b, :nk])
                x = s["q"][b, 0, h, a:e].double() @ k.T / math.sqrt(c["d"])
                minus = far.abs() * float(s["slopes"][h]) if c["slopes"] else None
                out[b, 0, h, a:e], lse[b, 0, h, a:e], _ = _row64(x, k, v, c["softcap"], minus, seen)
    return {"out": out, "lse": lse}


def _held64(codes, scale, d):
    """64-bit values of packed codes."""
    x = codes.long()
    low, high = x % 16, x // 16
    x = torch.stack((low - 16 * (low > 7), high - 16 * (high > 7)), -1).reshape(*codes.shape[:-1], d).double()
    return x * scale.double().repeat_interleave(d // scale.shape[-1], -1)


def _exact_attn(c, s):
    r, g, nq = s["rows"], c["heads"] // c["kv"], c["n_q"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    mass = r.mass.double()
    counts, nxt = r.count.tolist(), r.next_pos.tolist()
    for u in range(_units(c)):
        n, b, l, h0 = counts[u], u // (c["layers"] * c["kv"]), u // c["kv"] % c["layers"], u % c["kv"]
        k, v = _held64(r.k[u, :n], r.k_scale[u, :n], c["d"]), _held64(r.v[u, :n], r.v_scale[u, :n], c["d"])
        far = (torch.arange(nxt[u] - nq, nxt[u], device=DEV)[:, None] - r.pos[u, :n]).double()
        seen = (far >= 0) & ((far < c["window"]) if c["window"] else True)
        for h in range(h0 * g, h0 * g + g):
            if n == 0:
                lse[b, l, h] = -math.inf
                continue
            minus = far.abs() * float(s["slopes"][h]) if c["slopes"] else None
            x = s["q"][b, l, h].double() @ k.T / math.sqrt(c["d"])
            out[b, l, h], lse[b, l, h], w = _row64(x, k, v, c["softcap"], minus, seen)
            if c["mass"]:
                mass[u, :n] += w.sum(0)
    return {"out": out, "lse": lse, "mass": mass}


def _round64(x, mode):
    """64-bit x to the nearest scale of the mode, ties to even, as 64 bits."""
    bits, low = (8, -133) if mode == G32 else (11, -24)
    step = torch.exp2((torch.floor(torch.log2(x.clamp(min=1e-300))) - (bits - 1)).clamp(min=low))
    return torch.round(x / step) * step


def _stored64(x, mode):
    """64-bit values that bf16 rows have after 4 bits."""
    d = x.shape[-1]
    n = 32 if mode == G32 else d
    f = x.double().reshape(*x.shape[:-1], d // n, n)
    big = f.abs().max(-1, keepdim=True).values
    scale = _round64(big / 7, mode)
    scale = torch.where(big > 0, scale.clamp(min=2.0 ** (-133 if mode == G32 else -24)), 1.0)
    return (torch.round(f / scale).clamp(-7, 7) * scale).reshape(x.shape)


def _exact_store(c, s):
    live = torch.arange(c["n"], device=DEV) < _int(_new(c))[:, None]
    got = {x: torch.where(live[:, None, None, :, None], _stored64(s[x], c["mode"]), 0.0) for x in "kv"}
    return {**got, "pos": None, "counters": None}


def _exact_evict(c, s):
    """Units one after another on the host: sorted lists, row by row."""
    r, n, budget, u = s["rows"], c["n"], c["budget"], _units(c)
    pos, mass = r.pos.cpu().numpy().copy(), r.mass.cpu().numpy().copy()
    old = {x: _held64(getattr(r, x)[:, :budget], getattr(r, x + "_scale")[:, :budget], c["d"]) for x in "kv"}
    new = {x: _stored64(s[x].reshape(u, n, c["d"]), c["mode"]) for x in "kv"}
    src = np.zeros((u, budget), np.int64)
    nxt = r.next_pos.tolist()
    for i in range(u):
        pos[i, budget:] = np.arange(nxt[i], nxt[i] + n)
        mass[i, budget:] = 0
        free = np.nonzero((pos[i] >= N_SINK) & (pos[i] < nxt[i] + n - N_RECENT))[0]
        gone = free[np.lexsort((-pos[i][free], mass[i][free]))[:n]]
        stay = np.setdiff1d(np.arange(budget, budget + n), gone)
        src[i] = np.arange(budget)
        src[i, np.sort(gone[gone < budget])] = stay
        pos[i, :budget], mass[i, :budget] = pos[i, src[i]], mass[i, src[i]]
    at = torch.from_numpy(src).to(DEV)[..., None].expand(-1, -1, c["d"])
    got = {x: torch.cat((old[x], new[x]), 1).gather(1, at).view(s["k_out"].shape) for x in "kv"}
    return {"k": got["k"], "v": got["v"], "pos": None, "mass": torch.from_numpy(mass).double(), "counters": None}


def exact(case, seed):
    s, c = prepare(case, seed), dict(case)
    return {"prompt": _exact_prompt, "store": _exact_store, "attn": _exact_attn, "evict": _exact_evict}[c["op"]](c, s)
