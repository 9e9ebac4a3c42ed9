"""The 4-bit quantiser's quotients are those of IEEE division: the arithmetic over every mantissa (CPU), and the codes
and scales that kvc_i4_append stores over every bf16 magnitude of a group's maximum (GPU, against the oracle)."""
import numpy as np
import pytest
import torch

import oracle as o

G32, ROW = 0, 1
F = np.float32


def rounded_sum(a, b):
    """a + b, two float64 numbers, rounded once to float32: the float64 sum is made odd where it is not exact, so that
    its own rounding decides no tie."""
    s = a + b
    t = s - a
    err = (a - (s - t)) + (b - t)
    bits = s.view(np.int64)
    odd = (bits & 1) == 1
    # towards the exact value: one step away from zero or towards it
    away = (err > 0) == (s > 0)
    fixed = np.where((err != 0) & ~odd, np.where(away, bits | 1, bits - 1), bits).view(np.float64)
    return fixed.astype(F)


def fma(a, b, c):
    """float32 fma: the product of two float32 numbers is exact in float64."""
    return rounded_sum(a.astype(np.float64) * b.astype(np.float64), c.astype(np.float64))


def corrected_quotient(x, b, y):
    q0 = (x * y).astype(F)
    return fma(fma(q0, -b, x), y, q0)


def test_emulated_fma_rounds_once():
    """Against exact rational arithmetic, ties and near-ties among the cases."""
    from fractions import Fraction
    r = np.random.RandomState(1)
    a, b = (r.randint(1 << 23, 1 << 24, 400).astype(F) for _ in range(2))
    c = (r.randint(1 << 23, 1 << 24, 400) * 2.0 ** r.randint(-30, 60, 400)).astype(F) * r.choice([-1, 1], 400).astype(F)
    a[:100], b[:100] = F(1 << 23) + np.arange(100, dtype=F), F(1 << 23) + F(1)      # products near halves of a step of c
    c[:100] = F(2.0 ** 70)
    got = fma(a, b, c)
    for i in range(400):
        exact = Fraction(float(a[i])) * Fraction(float(b[i])) + Fraction(float(c[i]))
        cands = [got[i], np.nextafter(got[i], F(np.inf)), np.nextafter(got[i], F(-np.inf))]
        off = [abs(Fraction(float(v)) - exact) for v in cands]
        assert off[0] <= min(off[1:]), i
        if off[0] in off[1:]:                                  # a tie: the even one
            assert int(got[i].view(np.int32)) % 2 == 0


@pytest.mark.parametrize("bits", [7, 10], ids=["bf16", "fp16"])
@pytest.mark.parametrize("ulp", [-1, 0, 1])
def test_codes_are_those_of_ieee_division(bits, ulp):
    """Every bf16 mantissa over every mantissa of the scale's format, quotients up to 8, with the reciprocal one ulp off
    either way (the approximate reciprocal's bound): the rounded quotient is that of the IEEE quotient."""
    b = (1 + np.arange(1 << bits, dtype=F) / F(1 << bits))[:, None]
    y = (F(1) / b).astype(F)
    y = (y.view(np.int32) + ulp).view(F)
    for e in range(-4, 4):
        x = ((1 + np.arange(128, dtype=F) / F(128)) * F(2.0 ** e))[None, :]
        shape = np.broadcast(x, b).shape
        xx, bb, yy = (np.ascontiguousarray(np.broadcast_to(t, shape)) for t in (x, b, y))
        want = (xx / bb).astype(F)
        ok = want <= 7.5
        got = corrected_quotient(xx, bb, yy)
        assert np.array_equal(np.rint(got)[ok], np.rint(want)[ok])


def test_rounded_scales_are_those_of_ieee_division():
    """max / 7 by the reciprocal of 7, rounded to either scale format, for every positive finite bf16 maximum whose
    quotient is a normal number."""
    a = (np.arange(1, 0x7f80, dtype=np.uint32) << 16).view(F)
    a = a[a >= F(2.0 ** -123)]
    y = np.full_like(a, F(1) / F(7))
    assert y[0] == F(float.fromhex("0x1.24924ap-3"))           # the kernel's constant
    got, want = corrected_quotient(a, np.full_like(a, F(7)), y), (a / F(7)).astype(F)
    to_bf16 = lambda t: torch.from_numpy(t).to(torch.bfloat16).float().numpy()
    assert np.array_equal(to_bf16(got), to_bf16(want))
    with np.errstate(over="ignore"):
        assert np.array_equal(got.astype(np.float16), want.astype(np.float16))


@pytest.mark.gpu
@pytest.mark.parametrize("d, mode", [(128, G32), (64, G32), (128, ROW), (64, ROW)])
def test_append_stores_the_oracles_codes_for_every_maximum(d, mode):
    """Every positive finite bf16 maximum with every bf16 magnitude from a 32nd of it up to itself, both signs."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()
    import budgeted_kv_cache_gb300 as kvc
    group = 32 if mode == G32 else d
    others = group - 1
    top = np.arange(1, 0x7f80, dtype=np.int32)[:, None]         # bf16 bits of the maximum
    below = np.arange(-(-640 // others) * others, dtype=np.int32)[None, :]
    mag = np.maximum(top - below % 640, 0)                      # 5 binades and what a subnormal maximum leaves
    bits = mag | ((below & 1) << 15)
    bits = bits.reshape(top.shape[0], -1, others)
    x = np.concatenate([np.broadcast_to(top[:, :, None], bits.shape[:2] + (1,)), bits], -1).reshape(-1)
    assert len(x) >= 640 * (0x7f80 - 1)
    x = np.concatenate([x, np.zeros(-len(x) % d, np.int32)]).astype(np.uint16).reshape(-1, d)
    n = len(x)
    rows16 = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16).view(1, 1, 1, n, d)
    shape = kvc.make_shape(1, 1, 1, 1, d, 1)
    rows = kvc.I4Rows.allocate(shape, n, mode)
    kvc.kvc_i4_append(shape, rows, rows16, rows16)
    torch.cuda.synchronize()
    for i in range(0, n, 1 << 16):
        want, s = o.quantize((x[i:i + (1 << 16)].astype(np.uint32) << 16).view(F), 7, mode)
        want = o.pack_int4(want)
        for codes, scale in ((rows.k, rows.k_scale), (rows.v, rows.v_scale)):
            assert np.array_equal(codes[0, i:i + (1 << 16)].cpu().numpy(), want)
            assert np.array_equal(scale[0, i:i + (1 << 16)].float().cpu().numpy(), s)
