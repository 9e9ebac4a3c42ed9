"""64-bit attention with score modifiers, and how far a bf16 / fp32 kernel may be from it.

Rounding counts (u = 2^-24 for fp32, half a step of bf16 is 2^-8 of a value at most):
  * a logit: products of bf16 values are exact in fp32; a sum of d of them is off by at most d u of the
    sum of their magnitudes (in any order), scaling, cap, bias and the base-2 logarithm's factor add a
    few u of the logit's and the bias's magnitude and a few u of the cap: e_x below;
  * a weight exp(x - lse): relative error at most 2 e_x (its own logit's and the row statistic's) plus the
    exponential's 2^-22 and the sum's n u;
  * the value product: each weight is rounded to bf16 once (2^-8 of the weight), so the output moves by at
    most 2^-8 sum w |v|; the fp32 sum adds n u of the same; then one rounding to bf16, 2^-8 of the output.
"""
import math

import torch

U = 2.0 ** -24


def visible(p_q, p_k, window=0, prefix=0):
    """[n_q][n] mask from positions (64-bit integers)."""
    dist = p_q[:, None] - p_k[None, :]
    ok = dist >= 0
    if window:
        ok = ok & (dist < window)
    return ok | (p_k[None, :] < prefix)


def attend(q, k, v, scale, seen, dist, softcap=0.0, slope=None):
    """One head: q [n_q][d], k, v [n][d] in 64 bits; returns out, lse, w and the error bounds of out, lse, w."""
    n, d = k.shape
    if n == 0:
        z = torch.zeros(q.shape[0], d, dtype=torch.float64, device=q.device)
        lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
        w = torch.zeros(q.shape[0], 0, dtype=torch.float64, device=q.device)
        return z, lse, w, z, torch.zeros_like(lse), w
    live = seen.any(0)
    k = torch.where(live[:, None], k, torch.zeros_like(k))    # what nobody sees may hold any bits
    v = torch.where(live[:, None], v, torch.zeros_like(v))
    x = q @ k.T * scale
    e = (d + 4) * U * (q.abs() @ k.abs().T * scale) + 4 * U * x.abs()
    if softcap > 0:
        x = softcap * torch.tanh(x / softcap)
        e = e + 8 * U * softcap
    if slope is not None:
        x = x - slope * dist.abs()
        e = e + 4 * U * (slope * dist.abs()) + 4 * U * x.abs()
    x = x.masked_fill(~seen, -math.inf)
    e = torch.where(seen, e + 4 * U * x.abs(), torch.zeros_like(e))
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    out = w @ v
    worst = e.amax(-1)                                       # of the row's logits
    e_lse = worst + 2.0 ** -22 + n * U + 8 * U * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse).abs()
    e_w = w * (e + e_lse[:, None] + 2.0 ** -22)
    e_out = e_w @ v.abs() + (2.0 ** -8 + n * U) * (w @ v.abs()) + 2.0 ** -8 * out.abs()
    return out, lse, w, e_out, e_lse, e_w


def close(got, want, bound, what):
    """Every value within its bound (a bound's own rounding aside); infinities equal."""
    got, want = got.double(), want.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: infinities differ"
    ok = torch.isfinite(want)
    off = (got - want).abs()[ok] - 1.0001 * bound[ok]
    assert off.numel() == 0 or float(off.max()) <= 0, f"{what}: {float(off.max()):.3g} past its bound"
