"""Cases of the rotary positions and of drafted trees over the 4-bit cache: what they compute, in plain
torch operations, and the calls that a user's program makes of the library.

Operators (each `op` of a case is one pass of a program):
  tables  kvc_rope_tables: cosines and sines of every position, scaled for long contexts
  rope    kvc_rope: queries and keys rotated to their positions (or back), half or interleaved
          layout, part of the head
  tree    kvc_i4_tree_attn: attention of a tree of drafted tokens over the 4-bit cache and over
          the tree's own bf16 rows; outputs and row log-sum-exps
  commit  kvc_i4_tree_commit: the accepted path's softmax weights added to the cache's mass, its
          rows quantised into the cache
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
G32, ROW = 0, 1                       # a bf16 scale per 32 elements, or an fp16 scale per row
HALF, PAIRS = 0, 1                    # element i turns with i + rot / 2, or 2i with 2i + 1
PLAIN, LINEAR, BASE, TURNS, DIMS = 0, 1, 2, 3, 4      # how angles are scaled


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the tables of a 32K context, as trained
        _tables("tables_32k", rows=32768, rot=128, kind=PLAIN),
        # those of a million positions, slow angles stretched
        _tables("tables_1m", rows=1 << 20, rot=128, kind=TURNS, factor=32.0, base=500000.0),
        # one token of each of eight sequences, one layer: launch and latency
        _rope("rope_token", batch=8, heads=32, kv=8, d=128, n=1, rot=128),
        # a long prompt, one layer
        _rope("rope_prompt", batch=1, heads=32, kv=8, d=128, n=32768, rot=128),
        # a padded batch as a projection leaves it, a quarter of the head in pairs, turned back
        _rope("rope_pairs_back", batch=5, heads=12, kv=4, d=64, n=2047, rot=16, layout=PAIRS, inverse=True, ragged=True,
              store="token"),
        # a small tree over one sequence's budgeted cache, one layer
        _tree("tree_small", batch=1, heads=32, kv=8, d=128, n=13, cap=2304, lo=2048),
        # a tree over one long cache
        _tree("tree_long", batch=1, heads=32, kv=8, d=128, n=32, cap=131072, lo=100000),
        # a batch of trees of 64 nodes over 32K rows each
        _tree("tree_batch", batch=8, heads=32, kv=8, d=128, n=64, cap=32768, lo=20000),
        # padded trees of an odd head group, row scales, capped, distance bias, sliding window
        _tree("tree_mods", batch=6, heads=20, kv=4, d=64, n=37, cap=9001, lo=300, mode=ROW, softcap=30.0, slopes=True,
              window=4096, ragged=True),
        # the accepted tokens of one sequence, one layer
        _commit("commit_step", batch=1, layers=1, heads=32, kv=8, d=128, n=13, steps=4, cap=2304, lo=2048),
        # those of a batch, a whole model's layers, budgeted caches
        _commit("commit_layers", batch=2, layers=36, heads=32, kv=8, d=128, n=64, steps=7, cap=2304, lo=2048),
        # long caches of a batch with row scales
        _commit("commit_long", batch=8, layers=1, heads=24, kv=8, d=128, n=31, steps=5, cap=32768, lo=20000, mode=ROW,
                softcap=50.0),
    ]


def _tables(name, **kw):
    return {**dict(op="tables", rows=1, rot=128, base=10000.0, kind=PLAIN, factor=1.0, length=4096, low=1.0, high=32.0,
                   magnitude=1.0), **kw, **({"name": name} if name else {})}


def _rope(name, **kw):
    return {**dict(op="rope", batch=1, layers=1, heads=8, kv=8, d=128, n=1, rot=128, layout=HALF, inverse=False, ragged=False,
                   store="head", rows=32768), **kw, **({"name": name} if name else {})}


def _tree(name, **kw):
    return {**dict(op="tree", batch=1, layers=1, heads=8, kv=8, d=128, n=1, cap=256, lo=1, mode=G32, softcap=0.0, slopes=False,
                   window=0, ragged=False), **kw, **({"name": name} if name else {})}


def _commit(name, **kw):
    return {**dict(op="commit", batch=1, layers=1, heads=8, kv=8, d=128, n=1, steps=1, cap=256, lo=1, mode=G32, softcap=0.0,
                   slopes=False, window=0), **kw, **({"name": name} if name else {})}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "tree", "tree", "tree", "commit", "commit"])
    d, kv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "tables":
        kind = rng.choice([PLAIN, LINEAR, BASE, TURNS, DIMS])
        return _tables(None, rows=_log(rng, 16, 1 << 20), rot=16 * rng.randint(1, 8),
                       base=rng.choice([10000.0, 500000.0, 1e6]), kind=kind,
                       factor=1.0 if kind == PLAIN else round(rng.uniform(1.5, 40.0), 3), length=rng.choice([2048, 8192, 32768]),
                       magnitude=rng.choice([1.0, 1.2]))
    if op == "rope":
        n = _log(rng, 1, 32768)
        while n * kv * (group + 1) * d > 32768 * 40 * 128:
            n //= 2
        batch = max(1, min(16, _log(rng, 1, 16), (1 << 27) // (n * kv * (group + 1) * d)))
        return _rope(None, batch=batch, heads=kv * group, kv=kv, d=d, n=n, rot=16 * rng.randint(1, d // 16),
                     layout=rng.choice([HALF, PAIRS]), inverse=rng.random() < 0.3, ragged=rng.random() < 0.5,
                     store=rng.choice(["head", "token"]))
    mode, cap, n = rng.choice([G32, ROW]), _log(rng, 1, 131072), _log(rng, 1, 256)
    mods = dict(softcap=rng.choice([0.0, 0.0, 30.0]), slopes=rng.random() < 0.3,
                window=rng.choice([0, 0, _log(rng, 1, 65536)]))
    if op == "tree":
        while n > 1 and n * group * kv * cap > 64 * 256 * 32768:
            n //= 2
        batch = max(1, min(8, _log(rng, 1, 8), 64 * 256 * 32768 // (n * group * kv * cap), (1 << 21) // (kv * cap)))
        return _tree(None, batch=batch, heads=kv * group, kv=kv, d=d, n=n, cap=cap, lo=rng.randint(0, cap), mode=mode,
                     ragged=rng.random() < 0.5, **mods)
    n = min(n, 64)
    steps = min(n, rng.randint(1, 10))
    units = max(1, min(144, (1 << 20) // (cap + 64)))
    layers = max(1, min(36, _log(rng, 1, 36), units // kv))
    return _commit(None, batch=max(1, min(8, units // (kv * layers), rng.randint(1, 8))), layers=layers, heads=kv * group, kv=kv,
                   d=d, n=n, steps=steps, cap=cap, lo=rng.randint(0, cap), mode=mode, **mods)


# ------------------------------------------------------------------------------ shapes a case fixes

def _units(c):
    return c["batch"] * c["layers"] * c["kv"]


def _counts(c):
    """Rows in use of each sequence's units: the first has the most."""
    r = np.random.RandomState(c["cap"] * 5 + c["lo"])
    return [c["cap"]] + [int(r.randint(c["lo"], c["cap"] + 1)) for _ in range(c["batch"] - 1)]


def _sizes(c):
    """Rows (or nodes) of each sequence: n, or ragged with one full sequence."""
    r = np.random.RandomState(c["n"] * 11 + c["batch"])
    return [c["n"] if i == 0 or not c["ragged"] else int(r.randint(0, c["n"] + 1)) for i in range(c["batch"])]


def _row_bytes(c):
    """Codes and scales of one vector."""
    return c["d"] // 2 + (2 * (c["d"] // 32) if c["mode"] == G32 else 2)


def work(case):
    c = case
    if c["op"] == "tables":
        return {"bytes": 4 * c["rows"] * c["rot"], "flops": 0}
    if c["op"] == "rope":
        n = sum(_sizes(c))
        return {"bytes": n * ((c["heads"] + c["kv"]) * c["layers"] * 4 * c["d"] + 4 * c["rot"] + 4),
                "flops": n * (c["heads"] + c["kv"]) * c["layers"] * 3 * c["rot"]}
    g = c["heads"] // c["kv"]
    lead = c["layers"] * c["kv"]
    keys = [min(n, c["window"]) if c["window"] else n for n in _counts(c)]
    some = 4 if c["window"] or c["slopes"] else 0                          # positions
    if c["op"] == "tree":
        nodes = _sizes(c)
        keys = [k if n else 0 for k, n in zip(keys, nodes)]
        rows = sum(nodes) * c["layers"] * c["heads"]
        pairs = sum(k * n + n * (n + 1) // 2 for k, n in zip(keys, nodes)) * lead * g
        return {"bytes": sum(keys) * lead * (2 * _row_bytes(c) + some) + sum(nodes) * (lead * 4 * c["d"] + 4) +
                rows * (4 * c["d"] + 4), "flops": 4 * c["d"] * pairs}
    n = c["steps"]
    return {"bytes": sum(keys) * lead * (_row_bytes(c) + some + 8) +
            c["batch"] * lead * n * (4 * c["d"] + g * (2 * c["d"] + 4) + 2 * _row_bytes(c) + 4 * c["d"] + 8),
            "flops": 2 * c["d"] * g * n * (sum(keys) + c["batch"] * n) * lead}


# ------------------------------------------------------------------------------ inputs

Q_NORM = 2.0                          # logits of about 2 standard deviations: rows attend to few of many keys


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _slopes(heads):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], device=DEV)


def _tensor(g, c, heads):
    """A [B][L][H][n][d] tensor, stored head by head or token by token as a projection leaves it."""
    if c["store"] == "token":
        return _randn(g, c["batch"], c["layers"], c["n"], heads, c["d"]).transpose(2, 3)
    return _randn(g, c["batch"], c["layers"], heads, c["n"], c["d"])


class Rows:
    """The arrays of a 4-bit cache: codes, scales, positions, accumulated weight, rows in use."""

    def __init__(self, c, cap, g, counts):
        u, d, mode = _units(c), c["d"], c["mode"]
        e = lambda *s, dt: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
        ns, sdt = (d // 32, torch.bfloat16) if mode == G32 else (1, torch.float16)
        self.k, self.v = e(u, cap, d // 2, dt=torch.uint8), e(u, cap, d // 2, dt=torch.uint8)
        self.k_scale, self.v_scale = e(u, cap, ns, dt=sdt), e(u, cap, ns, dt=sdt)
        for codes, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            step = max(1, (1 << 27) // (cap * d))
            for a in range(0, u, step):
                x = torch.randn((min(step, u - a), cap, d), generator=g, device=DEV)
                codes[a:a + step], scale[a:a + step] = _quantise(x.to(torch.bfloat16), mode)
        gap = torch.randint(1, 4, (u, cap), generator=g, device=DEV)
        self.pos = (torch.cumsum(gap, 1) - gap[:, :1]).to(torch.int32)
        self.mass = torch.rand((u, cap), generator=g, device=DEV) * 4
        self.counters = e(2, u, dt=torch.int32)              # rows in use, next position
        self.count, self.next_pos = self.counters[0], self.counters[1]
        self.count.copy_(counts)
        last = self.pos.gather(1, (counts.long() - 1).clamp(min=0)[:, None])[:, 0]
        self.next_pos.copy_(torch.where(counts > 0, last + 1, torch.zeros_like(last)))


def _parents(g, c):
    """Parent of each node, [B][n]: mostly one of the last few nodes, -1 for those that follow the cache."""
    i = torch.arange(c["n"], device=DEV)
    back = 1 + torch.floor(torch.rand((c["batch"], c["n"]), generator=g, device=DEV) ** 2 * 6).long()
    return (i - back).clamp(min=-1).to(torch.int32)


def _path(parent, steps, g):
    """A path of each tree from a first node down, [B][steps] (nodes behind its end: 0), and its length."""
    want = torch.randint(1, steps + 1, (parent.shape[0],), generator=g, device=DEV).tolist()
    path, size = np.zeros((parent.shape[0], steps), np.int64), []
    for b, row in enumerate(parent.tolist()):
        chains = []
        for i, up in enumerate(row):
            chains.append((chains[up] if up >= 0 else []) + [i])
        longest = max(chains, key=len)[:min(want[b], steps)]
        path[b, :len(longest)] = longest
        size.append(len(longest))
    return _int(path.tolist()), _int(size)


def _shape(c, n):
    import budgeted_kv_cache_gb300 as kvc
    return kvc.make_shape(c["batch"], c["layers"], c["heads"], c["kv"], c["d"], n)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "tables":
        # angles differ with the base, so that inputs of another seed are others
        s["base"] = c["base"] * (1.0 + float(torch.rand((), generator=g, device=DEV)))
        s["cos"] = torch.zeros(c["rows"], c["rot"] // 2, device=DEV)
        s["sin"] = torch.zeros_like(s["cos"])
        if own:
            import budgeted_kv_cache_gb300 as kvc
            s["scaling"] = kvc.RopeScaling(c["kind"], c["factor"], c["length"], c["low"], c["high"], c["magnitude"])
        return s
    if c["op"] == "rope":
        s["q"], s["k"] = _tensor(g, c, c["heads"]), _tensor(g, c, c["kv"])
        s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
        angle = torch.arange(c["rows"], device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        s["cos"], s["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
        first = torch.randint(0, c["rows"] - c["n"] + 1, (c["batch"], 1), generator=g, device=DEV)
        s["pos"] = (first + torch.arange(c["n"], device=DEV)).to(torch.int32)
        s["size"] = _int(_sizes(c)) if c["ragged"] else None
        if own:
            s["shape"] = _shape(c, c["n"])
        return s
    counts = _int(_counts(c)).repeat_interleave(c["layers"] * c["kv"])
    lead, n, d = (c["batch"], c["layers"]), c["n"], c["d"]
    rows = s["rows"] = Rows(c, c["cap"] + c.get("steps", 0), g, counts)
    s["q"] = _randn(g, *lead, c["heads"], n, d) * Q_NORM
    s["k"], s["v"] = _randn(g, *lead, c["kv"], n, d), _randn(g, *lead, c["kv"], n, d)
    s["parent"] = _parents(g, c)
    s["slopes"] = _slopes(c["heads"]) if c["slopes"] else None
    s["lse"] = torch.zeros(*lead, c["heads"], n, device=DEV)
    if c["op"] == "tree":
        s["out"] = torch.zeros_like(s["q"])
        s["size"] = _int(_sizes(c)) if c["ragged"] else None
    else:
        s["path"], s["size"] = _path(s["parent"], c["steps"], g)
        s["k_out"] = torch.zeros(*lead, c["kv"], c["steps"], d, dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.zeros_like(s["k_out"])
        s["start"] = rows.counters.clone()
        # the log-sum-exps that the attention of the tree left for the path's nodes
        on = torch.arange(c["steps"], device=DEV) < s["size"][:, None]
        at = torch.where(on, s["path"].long(), n)[:, None, None, :].expand(*lead, c["heads"], -1)
        lse = torch.zeros(*lead, c["heads"], n + 1, device=DEV).scatter_(3, at, _path_scores(c, s)[2])
        s["lse"].copy_(lse[..., :n])
    if own:
        import budgeted_kv_cache_gb300 as kvc
        s["shape"] = _shape(c, c["cap"])
        s["cache"] = kvc.I4Rows(rows.k, rows.v, rows.k_scale, rows.v_scale, rows.pos, rows.count, rows.next_pos, rows.mass,
                                c["mode"])
        s["mods"] = kvc.ScoreMods(c["softcap"], s["slopes"], c["window"])
        if c["op"] == "tree":
            s["ws"] = torch.empty(max(256, kvc.kvc_i4_tree_attn_workspace_bytes(s["shape"], s["cache"], n)),
                                  dtype=torch.uint8, device=DEV)
    return s


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


def _values(codes, scale):
    """fp32 values that codes and scales stand for."""
    x = codes.to(torch.int32)
    x = torch.stack((x & 15, x >> 4), -1).flatten(-2)
    x = ((x ^ 8) - 8).float()
    return (x.unflatten(-1, (scale.shape[-1], -1)) * scale.float()[..., None]).flatten(-2)


def _angles(c, base):
    """Angle per position of each pair, in 64 bits: 1 / base^(2i / rot), scaled."""
    rot, kind, factor = c["rot"], c["kind"], c["factor"]
    if kind == BASE:
        base = base * factor ** (rot / (rot - 2.0))
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    theta = base ** (-2.0 * i / rot)
    if kind == LINEAR:
        return theta / factor
    if kind == TURNS:                 # pairs that turn often in the trained length stay, slow ones are stretched
        keep = ((c["length"] * theta / (2 * math.pi) - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        return theta * (keep + (1 - keep) / factor)
    if kind == DIMS:                  # the same, linear in i between the pairs that turn `high` and `low` times
        at = lambda turns: rot * math.log(c["length"] / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        first, last = max(math.floor(at(c["high"])), 0), min(math.ceil(at(c["low"])), rot - 1)
        keep = 1 - ((i - first) / max(last - first, 0.001)).clamp(0, 1)
        return theta * (keep + (1 - keep) / factor)
    return theta


def _plain_tables(c, s):
    angle = torch.arange(c["rows"], dtype=torch.float64, device=DEV)[:, None] * _angles(c, s["base"])
    s["cos"].copy_(torch.cos(angle) * c["magnitude"])
    s["sin"].copy_(torch.sin(angle) * c["magnitude"])
    return {"cos": s["cos"], "sin": s["sin"]}


def _plain_rope(c, s):
    rot = c["rot"]
    p = s["pos"].long()
    cos, sin = s["cos"][p][:, None, None], s["sin"][p][:, None, None]
    if c["inverse"]:
        sin = -sin
    live = None if s["size"] is None else (torch.arange(c["n"], device=DEV) < s["size"][:, None])[:, None, None, :, None]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = x.float()
        if c["layout"] == HALF:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin, y[..., rot:]), -1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), y[..., rot:]), -1)
        out.copy_(turned if live is None else torch.where(live, turned, out))
    return {"q": s["q_out"], "k": s["k_out"]}


def _ancestors(parent):
    """[B][n][n]: whether node j is i or above it, by doubling the steps up."""
    n = parent.shape[1]
    i = torch.arange(n, device=DEV)
    up = (parent.long()[:, :, None] == i).float() + torch.eye(n, device=DEV)
    for _ in range(max(1, (n - 1).bit_length())):
        up = (up @ up > 0).float()
    return up > 0


def _scores(c, q, k, slopes, far, seen):
    """Scores (-inf where not seen) of q [B,L,heads,n,d] over k [B,L,kv,T,d]: [B,L,kv,G,n,T]."""
    g = c["heads"] // c["kv"]
    n = q.shape[3]
    rows = q.float().unflatten(2, (c["kv"], g)).flatten(3, 4)
    x = (rows @ k.transpose(-1, -2)).unflatten(3, (g, n)) * (1 / math.sqrt(c["d"]))
    if c["softcap"] > 0:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    if slopes is not None:
        x = x - slopes.view(1, 1, c["kv"], g, 1, 1) * far.abs()
    return torch.where(seen, x, float("-inf"))


def _cached(c, s, p_q):
    """Distances to the cached rows and whether they are seen, [B,L,kv,1,n,cap]; p_q [B,L,kv,n]."""
    r = s["rows"]
    lead = (c["batch"], c["layers"], c["kv"])
    far = p_q[..., None] - r.pos.view(*lead, 1, -1)
    seen = (torch.arange(r.pos.shape[1], device=DEV) < r.count.view(*lead, 1, 1)).expand(far.shape)
    if c["window"]:
        seen = seen & (far < c["window"])
    return far.unsqueeze(3), seen.unsqueeze(3)


def _softmax(x):
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, m + torch.log(total), float("-inf"))
    return p / torch.where(total > 0, total, torch.ones_like(total)), lse


def _plain_tree(c, s):
    r, lead = s["rows"], (c["batch"], c["layers"], c["kv"])
    above = _ancestors(s["parent"])
    depth = above.sum(-1) - 1
    p_q = r.next_pos.view(*lead, 1) + depth[:, None, None]
    far, seen = _cached(c, s, p_q)
    x = _scores(c, s["q"], _values(r.k, r.k_scale).view(*lead, -1, c["d"]), s["slopes"], far, seen)
    far = depth[:, :, None] - depth[:, None, :]
    seen = above & (far < c["window"]) if c["window"] else above
    far, seen = far[:, None, None, None], seen[:, None, None, None]
    x = torch.cat((x, _scores(c, s["q"], s["k"].float(), s["slopes"], far, seen)), -1)
    v = torch.cat((_values(r.v, r.v_scale).view(*lead, -1, c["d"]), s["v"].float()), 3)
    p, lse = _softmax(x)
    out = (p.flatten(3, 4) @ v).view(s["out"].shape)
    live = torch.arange(c["n"], device=DEV) < (c["n"] if s["size"] is None else s["size"][:, None])
    live = live.expand(c["batch"], -1)[:, None, None]
    s["out"].copy_(torch.where(live[..., None], out, s["out"]))
    s["lse"].copy_(torch.where(live, lse.view(s["lse"].shape), s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _path_scores(c, s):
    """Scores of the path's nodes over the cached rows and over the path's rows, and their log-sum-exps."""
    r, lead, n = s["rows"], (c["batch"], c["layers"], c["kv"]), c["steps"]
    take = lambda x: x.gather(3, s["path"].long()[:, None, None, :, None].expand(*x.shape[:3], n, x.shape[4]))  # noqa: E731
    q, k, i = take(s["q"]), take(s["k"]), torch.arange(n, device=DEV)
    far, seen = _cached(c, s, r.next_pos.view(*lead, 1) + i)
    x = _scores(c, q, _values(r.k, r.k_scale).view(*lead, -1, c["d"]), s["slopes"], far, seen)
    far = i[:, None] - i
    seen = (far >= 0) & ((far < c["window"]) if c["window"] else True)
    y = _scores(c, q, k.float(), s["slopes"], far, seen)
    return x, y, torch.logsumexp(torch.cat((x, y), -1), -1).view(*lead[:2], c["heads"], n)


def _plain_commit(c, s):
    r, lead, n, u = s["rows"], (c["batch"], c["layers"], c["kv"]), c["steps"], _units(c)
    r.counters.copy_(s["start"])
    x, y, _ = _path_scores(c, s)
    on = torch.arange(n, device=DEV) < s["size"][:, None]
    lse = s["lse"].gather(3, s["path"].long()[:, None, None, :].expand(*lead[:2], c["heads"], -1))
    lse = lse.view(*lead, -1, n, 1)
    row_on = on[:, None, None, None, :, None]
    r.mass.add_(torch.where(row_on, torch.exp(x - lse), 0.0).sum((3, 4)).view(r.mass.shape))
    fresh = torch.where(row_on, torch.exp(y - lse), 0.0).sum((3, 4)).view(u, n)
    # the path's rows behind those in use
    size = s["size"].repeat_interleave(u // c["batch"])
    i = torch.arange(n, device=DEV)
    slot = r.count[:, None].long() + i
    live = i < size[:, None]
    at = lambda i, x: i.view(u, n, *[1] * (x.dim() - 2)).expand_as(x)  # noqa: E731
    put = lambda x, new: x.scatter_(1, at(slot, new), torch.where(at(live, new), new, x.gather(1, at(slot, new))))  # noqa: E731
    for x, codes, scale, out in ((s["k"], r.k, r.k_scale, s["k_out"]), (s["v"], r.v, r.v_scale, s["v_out"])):
        x = x.gather(3, s["path"].long()[:, None, None, :, None].expand(*lead, n, c["d"]))
        q, sc = _quantise(x.reshape(u, n, c["d"]), c["mode"])
        put(codes, q)
        put(scale, sc)
        out.copy_(torch.where(live[..., None], _values(q, sc), out.view(u, n, -1).float()).view(out.shape))
    put(r.pos, r.next_pos[:, None] + i.int())
    put(r.mass, fresh)
    r.counters.add_(size.int())
    return {"k": s["k_out"], "v": s["v_out"], "pos": r.pos, "mass": r.mass, "counters": r.counters}


# ------------------------------------------------------------------------------ the library's calls

def _own_tables(c, s):
    import budgeted_kv_cache_gb300 as kvc
    kvc.kvc_rope_tables(s["cos"], s["sin"], s["base"], scaling=s["scaling"])
    return {"cos": s["cos"], "sin": s["sin"]}


def _own_rope(c, s):
    import budgeted_kv_cache_gb300 as kvc
    kvc.kvc_rope(s["shape"], s["q"], s["k"], s["pos"], s["cos"], s["sin"], s["q_out"], s["k_out"], n_rows=s["size"],
                 rope_layout=c["layout"], rotary_dim=c["rot"], inverse=c["inverse"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_tree(c, s):
    import budgeted_kv_cache_gb300 as kvc
    kvc.kvc_i4_tree_attn(s["shape"], s["cache"], s["q"], s["k"], s["v"], s["parent"], s["out"], n_nodes=s["size"],
                         mods=s["mods"], row_lse=s["lse"], workspace=s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_commit(c, s):
    import budgeted_kv_cache_gb300 as kvc
    r = s["rows"]
    r.counters.copy_(s["start"])
    kvc.kvc_i4_tree_commit(s["shape"], s["cache"], s["k"], s["v"], s["path"], s["size"], q=s["q"], row_lse=s["lse"],
                           mods=s["mods"], k_out=s["k_out"], v_out=s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"], "pos": r.pos, "mass": r.mass, "counters": r.counters}


def run(state):
    c = state["case"]
    if own:
        return {"tables": _own_tables, "rope": _own_rope, "tree": _own_tree, "commit": _own_commit}[c["op"]](c, state)
    return {"tables": _plain_tables, "rope": _plain_rope, "tree": _plain_tree, "commit": _plain_commit}[c["op"]](c, state)


# ------------------------------------------------------------------------------ the definitions in 64 bits

def _exact_tables(c, s):
    """Pair by pair: the angle's turns, their whole part dropped, then cosine and sine."""
    cos = torch.zeros(c["rows"], c["rot"] // 2, dtype=torch.float64, device=DEV)
    sin = torch.zeros_like(cos)
    p = torch.arange(c["rows"], dtype=torch.float64, device=DEV)
    rot, base = c["rot"], s["base"]
    if c["kind"] == BASE:
        base *= c["factor"] ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = math.exp(-math.log(base) * 2 * i / rot)
        t = {PLAIN: 1.0, BASE: 1.0, LINEAR: 0.0}.get(c["kind"])
        if c["kind"] == TURNS:
            t = (c["length"] * f / math.tau - c["low"]) / (c["high"] - c["low"])
        if c["kind"] == DIMS:
            a, b = (rot * math.log(c["length"] / math.tau / w, base) / 2 for w in (c["high"], c["low"]))
            a, b = max(math.floor(a), 0), min(math.ceil(b), rot - 1)
            t = 1 - (i - a) / max(b - a, 1e-3)
        t = min(max(t, 0.0), 1.0)
        f = f * t + f / c["factor"] * (1 - t)
        turn = p * (f / math.tau)
        turn = (turn - torch.round(turn)) * math.tau
        cos[:, i], sin[:, i] = torch.cos(turn) * c["magnitude"], torch.sin(turn) * c["magnitude"]
    return {"cos": cos, "sin": sin}


def _exact_rope(c, s):
    """Every pair as a complex number times one of the table's."""
    way = torch.complex(s["cos"].double(), s["sin"].double())
    if c["inverse"]:
        way = way.conj()
    got, rot = {}, c["rot"]
    for name, heads in (("q", c["heads"]), ("k", c["kv"])):
        out = torch.zeros(s[name].shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(_sizes(c)):
            x = s[name][b, :, :, :n].double()
            y = x.clone()
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) if c["layout"] == HALF else \
                torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous())
            z = z * way[s["pos"][b, :n].long()]
            if c["layout"] == HALF:
                y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
            else:
                y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
            out[b, :, :, :n] = y
        got[name] = out
    return got


def _held64(codes, scale, d):
    """64-bit values of packed codes."""
    x = codes.long()
    low, high = x % 16, x // 16
    x = torch.stack((low - 16 * (low > 7), high - 16 * (high > 7)), -1).reshape(*codes.shape[:-1], d).double()
    return x * scale.double().repeat_interleave(d // scale.shape[-1], -1)


def _logits64(c, s, q, k, h, far, seen):
    x = q @ k.T / math.sqrt(c["d"])
    if c["softcap"] > 0:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    if c["slopes"]:
        x = x - far.abs().double() * float(s["slopes"][h])
    if c["window"]:
        seen = seen & (far < c["window"])
    return x.masked_fill(~seen, -math.inf)


def _spots(c):
    for b in range(c["batch"]):
        for l in range(c["layers"]):
            for g in range(c["kv"]):
                yield (b * c["layers"] + l) * c["kv"] + g, b, l, g


def _exact_tree(c, s):
    r, group, d = s["rows"], c["heads"] // c["kv"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    counts, nxt, sizes, parents = r.count.tolist(), r.next_pos.tolist(), _sizes(c), s["parent"].tolist()
    for u, b, l, g in _spots(c):
        n, m = counts[u], sizes[b]
        if m == 0:
            continue
        lines = []                                    # every node's way up
        for i in range(m):
            up = parents[b][i]
            lines.append(([] if up < 0 else lines[up]) + [i])
        seen = torch.zeros(m, m, dtype=torch.bool)
        for i, line in enumerate(lines):
            seen[i, line] = True
        at = torch.tensor([nxt[u] + len(line) - 1 for line in lines], device=DEV)
        places = torch.cat((r.pos[u, :n].long(), at))
        seen = torch.cat((torch.ones(m, n, dtype=torch.bool, device=DEV), seen.to(DEV)), 1)
        k = torch.cat((_held64(r.k[u, :n], r.k_scale[u, :n], d), s["k"][b, l, g, :m].double()))
        v = torch.cat((_held64(r.v[u, :n], r.v_scale[u, :n], d), s["v"][b, l, g, :m].double()))
        for h in range(g * group, (g + 1) * group):
            x = _logits64(c, s, s["q"][b, l, h, :m].double(), k, h, at[:, None] - places, seen)
            lse[b, l, h, :m] = torch.logsumexp(x, -1)
            out[b, l, h, :m] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}


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


def _exact_commit(c, s):
    r, group, d = s["rows"], c["heads"] // c["kv"], c["d"]
    mass = r.mass.double()
    got = {x: torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEV) for x in "kv"}
    counts, nxt, paths, sizes = r.count.tolist(), r.next_pos.tolist(), s["path"].tolist(), s["size"].tolist()
    for u, b, l, g in _spots(c):
        n, line = counts[u], paths[b][:sizes[b]]
        m = len(line)
        new = s["k"][b, l, g, line]
        k = torch.cat((_held64(r.k[u, :n], r.k_scale[u, :n], d), new.double()))
        at = torch.arange(nxt[u], nxt[u] + m, device=DEV)
        far = at[:, None] - torch.cat((r.pos[u, :n].long(), at))
        seen = torch.cat((torch.ones(m, n, dtype=torch.bool, device=DEV),
                          torch.ones(m, m, dtype=torch.bool, device=DEV).tril()), 1)
        total = torch.zeros(n + m, dtype=torch.float64, device=DEV)
        for h in range(g * group, (g + 1) * group):
            x = _logits64(c, s, s["q"][b, l, h, line].double(), k, h, far, seen)
            total += torch.exp(x - s["lse"][b, l, h, line].double()[:, None]).sum(0)
        mass[u, :n] += total[:n]
        mass[u, n:n + m] = total[n:]
        got["k"][b, l, g, :m] = _stored64(new, c["mode"])
        got["v"][b, l, g, :m] = _stored64(s["v"][b, l, g, line], c["mode"])
    return {"k": got["k"], "v": got["v"], "pos": None, "mass": mass, "counters": None}


def exact(case, seed):
    s, c = prepare(case, seed), dict(case)
    return {"tables": _exact_tables, "rope": _exact_rope, "tree": _exact_tree, "commit": _exact_commit}[c["op"]](c, s)
