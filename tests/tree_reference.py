"""Trees of drafted tokens over a 4-bit cache in 64 bits, and how far a kernel may be from them: the bounds of
attn_reference, but for a weight's rounding, which is fp16's half step at most, and one more of the output.

A weight is held in fp16 or finer, relative to the largest product of a weight and its tile's largest value:
P'' = 2^(y + e - M) with M within the maximum of y + e, 2^e the size of the tile's values.  Below 2^-14 fp16 has
steps of 2^-24 (below 2^-126 fp32 has none), so P'' is off by at most 2^-25 there, and the output by 2^-25 of a
product 2^(M - L) V' <= max_j w_j max|v|, L the row's log-sum-exp: at most n 2^-25 max|v| over n keys."""
import numpy as np
import torch

import oracle as o
from attn_reference import U, attend


def held(codes, scale, d):
    """64-bit values of packed rows."""
    c = torch.from_numpy(o.unpack_int4(codes.cpu().numpy()).astype(np.float64)).to(codes.device)
    return c * scale.double().repeat_interleave(d // scale.shape[-1], -1)


def lines(parent):
    """Every node's way down to itself, first node first."""
    out = []
    for i, p in enumerate(parent):
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


def trees(kind, n, seed=0):
    """Parents of n nodes."""
    r = np.random.RandomState(seed + n)
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "roots":
        return [-1] * n
    return [int(r.randint(max(-1, i - 9), i)) if i else -1 for i in range(n)]


def heads_of(rows, u, q, k_new, v_new, parent, scale, softcap=0.0, slopes=None, window=0, prefix=-2 ** 40):
    """One unit: q [G][n][d], k_new, v_new [n][d] (64 bits, nodes only): what attend gives for each head, and the values."""
    G, n, d = q.shape
    count, nxt = int(rows.count[u]), int(rows.next_pos[u])
    way = lines(parent)
    at = torch.tensor([nxt + len(w) - 1 for w in way], dtype=torch.int64, device=q.device)
    pos = torch.cat((rows.pos[u, :count].long(), at))
    seen = torch.zeros(n, n, dtype=torch.bool)
    for i, w in enumerate(way):
        seen[i, w] = True
    seen = torch.cat((torch.ones(n, count, dtype=torch.bool, device=q.device), seen.to(q.device)), 1)
    dist = at[:, None] - pos
    if window:
        seen = seen & ((dist < window) | (pos < prefix))
    k = torch.cat((held(rows.k[u, :count], rows.k_scale[u, :count], d), k_new))
    v = torch.cat((held(rows.v[u, :count], rows.v_scale[u, :count], d), v_new))
    return [attend(q[h], k, v, scale, seen, dist, softcap, None if slopes is None else float(slopes[h])) for h in range(G)], v


def tree_attention(rows, u, q, k_new, v_new, parent, scale, **mods):
    """out, lse and their bounds, [G][n]."""
    got, v = heads_of(rows, u, q, k_new, v_new, parent, scale, **mods)
    got = [torch.stack([x[i] for x in got]) for i in range(5)]
    got[3] = got[3] + v.shape[0] * 2.0 ** -25 * v.abs().max() - (2.0 ** -8 - 2.0 ** -11) * (got[2] @ v.abs())
    return got


def path_mass(rows, u, q, k_new, scale, **mods):
    """Of a path (q [G][m][d], k_new [m][d]): log-sum-exps [G][m], the weight that every cached and path row gets from
    its queries, and how far a sum of fp32 weights may be from it (in any order)."""
    m = q.shape[1]
    got, _ = heads_of(rows, u, q, k_new, k_new, list(range(-1, m - 1)), scale, **mods)
    w = sum(x[2].sum(0) for x in got)
    return torch.stack([x[1] for x in got]), w, sum(x[5].sum(0) for x in got) + (len(got) * m + 8) * U * w
