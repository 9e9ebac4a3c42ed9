"""The tanh cap over its whole range of values, in kvc_prompt_attn and kvc_i4_attn: caps far above the scores (which
they leave nearly as they are), caps near zero (which make every score alike), small softmax scales, and rows whose
scores pass the cap beside rows that stay far below it.

Errors of a capped logit x = c tanh(z), z = s scale / c (u = 2^-24, S = sum |q||k| scale): the product is off by at
most (d + 4) u S.  Where |z| <= 0.625 a polynomial is used: its own error of 2.2e-7 = 3.7 u of the value, one rounding
each of z, z^2, the leading coefficient (2), the last step of the Horner chain (the ones before count by z^2 < 0.4) and
the product: below 16 u |x|.  Elsewhere c (1 - 2 / (1 + e^2z)) costs at most 2 c (1 - r) r (6 |z| + 4) u + 2 c r 3 u with
r = 1 / (1 + e^2z) (2^-22 of the exponential, 2^-23 of the reciprocal, the argument's roundings) and two roundings of
x, which is below 8 u c + 16 u |x|.  That form may stand for every score up to caps of 1,024, and for scores past 0.6 c
alone above.  Weights, sums and outputs as in attn_reference, and a weight below 2^-126 of the row's largest one may become
zero (the exponential's smallest result; the sum is at least one largest weight): 2^-126 a weight, and as much again for
the product's and the output's own steps below bf16's smallest normal value, 2^-134 each.
"""
import math

import pytest
import torch

from attn_reference import U, close, visible
from test_gpu_i4_cache import G32, ROW, Cache, held, randn
from test_gpu_prompt_attn import Case

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


def attend_capped(q, k, v, scale, seen, dist, cap, slope):
    """One head in 64 bits: out, lse, w and their bounds."""
    n, d = k.shape
    live = seen.any(0)
    k, v = (torch.where(live[:, None], t, torch.zeros_like(t)) for t in (k, v))
    s = q @ k.T * scale
    x = cap * torch.tanh(s / cap)
    e = (d + 4) * U * (q.abs() @ k.abs().T * scale) + 16 * U * x.abs()
    e = e + 8 * U * cap * ((s.abs() > 0.6 * cap) | (cap <= 1024)).double()
    if slope is not None:
        x = x - slope * dist.abs()
        e = e + 4 * U * (slope * dist.abs())
    x = x.masked_fill(~seen, -math.inf)
    e = torch.where(seen, e + 8 * U * x.abs(), torch.zeros_like(e))
    lse = torch.logsumexp(x, -1)
    flat = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
    w = torch.exp(x - flat[:, None])
    out = w @ v
    # a row's statistic is off by the weighted mean of its logits' errors at most (their second order aside)
    e_lse = (w * torch.expm1(e)).sum(-1) + 2.0 ** -22 + n * U + 8 * U * flat.abs()
    e_w = w * (torch.expm1(e) + torch.expm1(e_lse)[:, None] + 2.0 ** -22) + 2.0 ** -125
    e_out = e_w @ v.abs() + (2.0 ** -8 + n * U) * (w @ v.abs()) + 2.0 ** -8 * out.abs()
    return out, lse, w, e_out, e_lse, e_w


def check_prompt(c):
    torch.cuda.synchronize()
    scale = c.scale or 1 / math.sqrt(c.d)
    cap = float(torch.tensor(c.softcap, dtype=torch.float32))
    for b in range(c.B):
        nk = c.T if c.kv_len is None else int(c.kv_len[b])
        nq = c.n_q if c.q_len is None else int(c.q_len[b])
        p_q, p_k = torch.arange(nk - nq, nk, device="cuda"), torch.arange(nk, device="cuda")
        seen = visible(p_q, p_k, c.window, 0 if c.prefix is None else int(c.prefix[b]))
        if c.docs is not None:
            d = c.docs[b, :nk]
            seen = seen & (d[p_q][:, None] == d[None, :]) & (d >= 0)[None, :]
        dist = (p_q[:, None] - p_k[None, :]).double()
        for h in range(c.Hkv * c.G):
            k, v = c.k[b, 0, h // c.G, :nk].double(), c.v[b, 0, h // c.G, :nk].double()
            o, lse, _, e_o, e_l, _ = attend_capped(c.q[b, 0, h, :nq].double(), k, v, scale, seen, dist, cap,
                                                   None if c.slopes is None else float(c.slopes[h]))
            close(c.out[b, 0, h, :nq], o, e_o, f"out b{b} h{h}")
            close(c.lse[b, 0, h, :nq], lse, e_l, f"lse b{b} h{h}")


FORMS = {
    "causal": dict(n_q=200, T=200),
    "chunk": dict(n_q=70, T=333, G=3),
    "window": dict(n_q=150, T=300, window=40),
    "docs": dict(n_q=300, T=300, docs=[0] * 130 + [-1] * 20 + [1] * 150),
    "ragged": dict(B=2, n_q=150, T=400, q_len=[150, 31], kv_len=[390, 141]),
    "slopes": dict(n_q=140, T=260, slopes=True, prefix=[100]),
    "one_token": dict(n_q=1, T=5000),
}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("cap", [1e3, 1e4, 2e4, 1e6, 1e30, 3e38])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_caps_far_above_the_scores(kvc, d, cap, form):
    c = Case(kvc, d=d, softcap=cap, **FORMS[form])
    c.run()
    check_prompt(c)


@pytest.mark.parametrize("scale, cap", [(1e-4, 50.0), (1 / 128, 2000.0), (1e-10, 1.0), (1e-3, 30.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_small_scales(kvc, d, scale, cap):
    c = Case(kvc, d=d, n_q=200, T=200, softcap=cap, scale=scale, q_norm=30.0)
    c.run()
    check_prompt(c)


@pytest.mark.parametrize("cap", [1e-2, 1e-6, 1e-12, 1e-30, 1e-42])
@pytest.mark.parametrize("form", ["causal", "slopes"])
def test_prompt_caps_near_zero(kvc, cap, form):
    """Rows of zero scores among them: no coefficient may overflow into 0 times infinity."""
    c = Case(kvc, softcap=cap, **FORMS[form])
    c.q[:, :, :, ::5] = 0
    c.k[:, :, :, 60:] = 0
    c.run()
    check_prompt(c)


@pytest.mark.parametrize("cap", [30.0, 1e3, 5e3, 3e4])
@pytest.mark.parametrize("form", ["causal", "slopes", "window"])
def test_prompt_rows_past_the_cap_beside_rows_far_below(kvc, cap, form):
    """Every 16th query's scores reach the cap; its neighbours' stay of ordinary size and as accurate."""
    c = Case(kvc, softcap=cap, **FORMS[form])
    c.q[:, :, :, ::16].mul_(cap)
    c.run()
    check_prompt(c)


def i4_case(kvc, cap, mode, d, n_q, slopes, window, big, zeros):
    c = Cache(kvc, 2, 1, 2, d, 300, [300, 77], mode, 5, 8)
    q = randn(c.g, 2, 1, 8, n_q, d).mul_(2)
    if big:
        q[:, :, ::3].mul_(cap)
    if zeros:
        q[:, :, ::3] = 0
    sl = torch.rand(8, generator=c.g, device="cuda") * 0.01 if slopes else None
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:-1], 9.0, device="cuda")
    ws = torch.empty(max(1, kvc.kvc_i4_attn_workspace_bytes(c.shape, c.rows, n_q, True)), dtype=torch.uint8, device="cuda")
    c.rows.mass.zero_()
    kvc.kvc_i4_attn(c.shape, c.rows, q, out, mods=kvc.ScoreMods(cap, sl, window), add_mass=True, row_lse=lse, workspace=ws)
    torch.cuda.synchronize()
    cap = float(torch.tensor(cap, dtype=torch.float32))
    for u in range(4):
        b, g, n = u // 2, u % 2, int(c.rows.count[u])
        k, v = held(c.rows.k[u, :n], c.rows.k_scale[u, :n], d), held(c.rows.v[u, :n], c.rows.v_scale[u, :n], d)
        p_q = int(c.rows.next_pos[u]) - n_q + torch.arange(n_q, device="cuda")
        p_k = c.rows.pos[u, :n].long()
        seen = visible(p_q, p_k, window, -1)
        mass, e_mass = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
        for h in range(g * 4, g * 4 + 4):
            o, l, w, e_o, e_l, e_w = attend_capped(q[b, 0, h].double(), k, v, 1 / math.sqrt(d), seen,
                                                   (p_q[:, None] - p_k[None]).double(), cap,
                                                   None if sl is None else float(sl[h]))
            close(out[b, 0, h], o, e_o, f"out u{u} h{h}")
            close(lse[b, 0, h], l, e_l, f"lse u{u} h{h}")
            mass += w.sum(0)
            e_mass += e_w.sum(0) + 4 * n_q * U * w.sum(0)
        close(c.rows.mass[u, :n], mass, e_mass + U * mass, f"mass u{u}")


@pytest.mark.parametrize("cap", [1e3, 2e4, 1e6, 1e30, 3e38, 1e-2, 1e-12, 1e-30, 1e-42])
@pytest.mark.parametrize("mode, d, n_q", [(G32, 128, 1), (ROW, 64, 3), (G32, 64, 9)])
def test_4_bit_caps_far_from_the_scores(kvc, mode, d, n_q, cap):
    for slopes, window in ((False, 0), (True, 120)):
        i4_case(kvc, cap, mode, d, n_q, slopes, window, False, cap < 1)


@pytest.mark.parametrize("cap", [30.0, 1e3, 5e3, 3e4])
@pytest.mark.parametrize("mode, d, n_q", [(G32, 128, 1), (ROW, 64, 3), (G32, 64, 9)])
def test_4_bit_rows_past_the_cap_beside_rows_far_below(kvc, mode, d, n_q, cap):
    for slopes, window in ((False, 0), (True, 120)):
        i4_case(kvc, cap, mode, d, n_q, slopes, window, True, False)
