"""kvc_rope_tables and kvc_rope against their definitions (GPU)."""
import math

import pytest
import torch

import budgeted_kv_cache_gb300 as kvc

pytestmark = pytest.mark.gpu
HALF, PAIRS = kvc.ROPE_SPLIT_HALF, kvc.ROPE_INTERLEAVED


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()


def angles(rot, base, s):
    """Angle per position of each pair, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if s.kind == kvc.ROPE_SCALE_BASE:
        base = base * s.factor ** (rot / (rot - 2))
    theta = base ** (-2 * i / rot)
    keep = torch.ones_like(theta)
    if s.kind == kvc.ROPE_SCALE_LINEAR:
        keep = torch.zeros_like(theta)
    elif s.kind == kvc.ROPE_SCALE_TURNS:
        keep = ((s.original_len * theta / (2 * math.pi) - s.low) / (s.high - s.low)).clamp(0, 1)
    elif s.kind == kvc.ROPE_SCALE_DIMS:
        at = lambda n: rot * math.log(s.original_len / (2 * math.pi * n)) / (2 * math.log(base))
        a, b = max(math.floor(at(s.high)), 0), min(math.ceil(at(s.low)), rot - 1)
        keep = 1 - ((i - a) / max(b - a, 0.001)).clamp(0, 1)
    return theta * (keep + (1 - keep) / s.factor)


SCALINGS = [kvc.RopeScaling(), kvc.RopeScaling(kvc.ROPE_SCALE_LINEAR, 8.0), kvc.RopeScaling(kvc.ROPE_SCALE_LINEAR, 0.05),
            kvc.RopeScaling(kvc.ROPE_SCALE_BASE, 4.0), kvc.RopeScaling(kvc.ROPE_SCALE_TURNS, 32.0, 8192.0, 1.0, 4.0),
            kvc.RopeScaling(kvc.ROPE_SCALE_TURNS, 4.0, 100.0, 0.0, 0.5, -2.5),
            kvc.RopeScaling(kvc.ROPE_SCALE_DIMS, 16.0, 4096.0, 1.0, 32.0, 0.1 * math.log(16.0) + 1)]


@pytest.mark.parametrize("s", SCALINGS, ids=range(len(SCALINGS)))
@pytest.mark.parametrize("rot", [16, 48, 112, 128])
@pytest.mark.parametrize("n,base", [(1, 1e4), (17, 1.0), (3001, 1e4), (140001, 5e5)])
def test_tables(s, rot, n, base):
    if s.kind == kvc.ROPE_SCALE_DIMS and base == 1.0:
        base = 1e4
    cos, sin = torch.full((n, rot // 2), 9.0, device="cuda"), torch.full((n, rot // 2), 9.0, device="cuda")
    kvc.kvc_rope_tables(cos, sin, base, s)
    x = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * angles(rot, base, s).cuda()
    # the documented bound: polynomials within 1e-7, a 32-bit angle (2^-33 turns), the magnitude's rounding
    for got, want in ((cos, torch.cos(x)), (sin, torch.sin(x))):
        assert float((got.double() - want * s.magnitude).abs().max()) <= 2.0 ** -22 * abs(s.magnitude)


def test_tables_of_far_positions():
    """50 million positions: angles past what fp32 (and fp32 products) can tell apart."""
    n, rot = 50_000_000, 16
    cos, sin = torch.empty(n, rot // 2, device="cuda"), torch.empty(n, rot // 2, device="cuda")
    kvc.kvc_rope_tables(cos, sin, 10000.0)
    at = torch.cat((torch.arange(n - 70000, n), torch.randint(0, n, (70000,), generator=torch.Generator().manual_seed(1)))).cuda()
    x = at.double()[:, None] * angles(rot, 10000.0, kvc.RopeScaling()).cuda()
    # the definition's own product is off by 2^-53 of the angle, 50e6 2^-53 = 6e-9
    assert float((cos[at].double() - torch.cos(x)).abs().max()) <= 2.0 ** -22 + 1e-8
    assert float((sin[at].double() - torch.sin(x)).abs().max()) <= 2.0 ** -22 + 1e-8


def rotated(x, pos, cos, sin, layout, rot, inverse):
    """The same products and sums in fp32, one operation at a time."""
    y = x.float()
    c, s = cos[pos.long()][:, None, None], sin[pos.long()][:, None, None]
    if inverse:
        s = -s
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if layout == HALF else (y[..., 0:rot:2], y[..., 1:rot:2])
    u, v = a * c - b * s, b * c + a * s
    z = torch.cat((u, v), -1) if layout == HALF else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((z, y[..., rot:]), -1).to(torch.bfloat16)


def make(B, L, H, n, d, by_token, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if by_token:
        return torch.randn(B, L, n, H, d, generator=g, device="cuda").to(torch.bfloat16).transpose(2, 3)
    return torch.randn(B, L, H, n, d, generator=g, device="cuda").to(torch.bfloat16)


def tables(n, rot):
    x = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * angles(rot, 1e4, kvc.RopeScaling()).cuda()
    return torch.cos(x).float(), torch.sin(x).float()


CASES = [  # B, L, Hq, Hkv, d, n, rot, layout, by_token, inverse
    (1, 1, 1, 1, 128, 1, 128, HALF, False, False),
    (8, 1, 32, 8, 128, 1, 128, HALF, False, False),
    (3, 2, 12, 4, 64, 2, 64, PAIRS, True, False),
    (2, 3, 5, 5, 64, 33, 48, HALF, True, True),
    (1, 1, 32, 8, 128, 1000, 128, PAIRS, False, True),
    (2, 1, 7, 1, 128, 31, 16, HALF, False, False),
    (2, 1, 7, 1, 128, 31, 112, PAIRS, True, False),
    (1, 2, 9, 3, 64, 4097, 32, HALF, True, False),
    (5, 1, 64, 1, 128, 65, 96, PAIRS, False, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("in_place", [False, True])
def test_rotation(case, in_place):
    B, L, Hq, Hkv, d, n, rot, layout, by_token, inverse = case
    shape = kvc.make_shape(B, L, Hq, Hkv, d, 1)
    q, k = make(B, L, Hq, n, d, by_token, 1), make(B, L, Hkv, n, d, not by_token, 2)
    cos, sin = tables(5000, rot)
    pos = torch.randint(0, 5000, (B, n), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda", dtype=torch.int32)
    want_q, want_k = (rotated(x, pos, cos, sin, layout, rot, inverse) for x in (q, k))
    status = torch.full((B * L * Hkv,), 77, dtype=torch.int32, device="cuda")
    q_out, k_out = (None, None) if in_place else (make(B, L, Hq, n, d, not by_token, 5), make(B, L, Hkv, n, d, not by_token, 6))
    kvc.kvc_rope(shape, q, k, pos, cos, sin, q_out, k_out, rope_layout=layout, rotary_dim=rot, inverse=inverse, unit_status=status)
    got_q, got_k = (q, k) if in_place else (q_out, k_out)
    assert torch.equal(got_q, want_q) and torch.equal(got_k, want_k)
    assert (status == 77).all()


@pytest.mark.parametrize("which", ["q", "k"])
def test_one_of_both_and_padded_batches(which):
    B, L, H, n, d = 4, 2, 6, 19, 64
    shape = kvc.make_shape(B, L, H, H, d, 1)
    x = make(B, L, H, n, d, False, 1)
    cos, sin = tables(100, d)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B, 1)
    size = torch.tensor([n, 0, 7, 1000], dtype=torch.int32, device="cuda")
    pos[2, 7:] = -5                                            # not read
    out = make(B, L, H, n, d, True, 2)
    before, status = out.clone(), torch.zeros(B * L * H, dtype=torch.int32, device="cuda")
    args = (x, None) if which == "q" else (None, x)
    outs = (out, None) if which == "q" else (None, out)
    kvc.kvc_rope(shape, *args, pos, cos, sin, *outs, n_rows=size, unit_status=status)
    want = rotated(x, pos.clamp(min=0), cos, sin, HALF, d, False)
    live = (torch.arange(n, device="cuda") < size[:, None])[:, None, None, :, None]
    assert torch.equal(out, torch.where(live, want, before))
    assert int(status.abs().sum()) == 0


def test_positions_outside_the_tables_are_left_and_marked():
    B, L, Hq, Hkv, n, d = 3, 2, 4, 2, 11, 128
    shape = kvc.make_shape(B, L, Hq, Hkv, d, 1)
    q, k = make(B, L, Hq, n, d, False, 1), make(B, L, Hkv, n, d, False, 2)
    cos, sin = tables(50, 64)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B, 1)
    pos[0, 3], pos[2, 10], pos[2, 0] = -1, 50, 2 ** 31 - 1
    q_out, k_out = make(B, L, Hq, n, d, False, 3), make(B, L, Hkv, n, d, False, 4)
    bad = (pos < 0) | (pos >= 50)
    want = [torch.where(bad[:, None, None, :, None], o, rotated(x, pos.clamp(0, 49), cos, sin, PAIRS, 64, False))
            for x, o in ((q, q_out), (k, k_out))]
    status = torch.zeros(B, L, Hkv, dtype=torch.int32, device="cuda")
    kvc.kvc_rope(shape, q, k, pos, cos, sin, q_out, k_out, rope_layout=PAIRS, rotary_dim=64, unit_status=status)
    assert torch.equal(q_out, want[0]) and torch.equal(k_out, want[1])
    assert status.tolist() == [[[2, 2]] * 2, [[0, 0]] * 2, [[2, 2]] * 2]


@pytest.mark.parametrize("layout", [HALF, PAIRS])
def test_turning_back_is_the_gradient(layout):
    """<R x, y> = <x, R^T y> with R^T = R_-p; and the difference of R along a direction is R of the direction."""
    shape = kvc.make_shape(1, 1, 3, 3, 64, 1)
    x, y = make(1, 1, 3, 50, 64, False, 1), make(1, 1, 3, 50, 64, False, 2)
    cos, sin = tables(2000, 48)
    pos = torch.randint(0, 2000, (1, 50), device="cuda", dtype=torch.int32)
    rx, ry = x.clone(), y.clone()
    kvc.kvc_rope(shape, rx, None, pos, cos, sin, rope_layout=layout, rotary_dim=48)
    kvc.kvc_rope(shape, ry, None, pos, cos, sin, rope_layout=layout, rotary_dim=48, inverse=True)
    a, b = (rx.double() * y.double()).sum(), (x.double() * ry.double()).sum()
    # every element of R x and R^T y is off by at most 2^-8 of itself, plus 2^-22 of its pair's magnitudes
    slack = (2.0 ** -8 + 2.0 ** -21) * ((rx.double() * y.double()).abs().sum() + (x.double() * ry.double()).abs().sum())
    assert abs(float(a - b)) <= float(slack)
    # differences: x + h e and x - h e with powers of two, so that the inputs are exact
    e = torch.randint(0, 2, x.shape, device="cuda").to(torch.bfloat16) * 2 - 1
    up, down, way = e * 8, e * -8, e.clone()
    for t in (up, down, way):
        kvc.kvc_rope(shape, t, None, pos, cos, sin, rope_layout=layout, rotary_dim=48)
    diff = (up.double() - down.double()) / 16
    assert float((diff - way.double()).abs().max()) <= 2 * 2.0 ** -8 * 1.4143


def test_capture_and_other_streams():
    shape = kvc.make_shape(2, 1, 8, 2, 128, 1)
    q, k = make(2, 1, 8, 9, 128, False, 1), make(2, 1, 2, 9, 128, False, 2)
    pos = torch.arange(9, dtype=torch.int32, device="cuda").repeat(2, 1)
    cos, sin = torch.empty(64, 64, device="cuda"), torch.empty(64, 64, device="cuda")
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        kvc.kvc_rope_tables(cos, sin)
        kvc.kvc_rope(shape, q, k, pos, cos, sin, q_out, k_out)
    side.synchronize()
    want = [rotated(x, pos, cos, sin, HALF, 128, False) for x in (q, k)]
    assert torch.equal(q_out, want[0]) and torch.equal(k_out, want[1])
    with torch.cuda.graph(graph):
        kvc.kvc_rope_tables(cos, sin, 500000.0)
        kvc.kvc_rope(shape, q, k, pos, cos, sin, q_out, k_out)
    for _ in range(2):
        pos += 3
        graph.replay()
        torch.cuda.synchronize()
        want = [rotated(x, pos, cos, sin, HALF, 128, False) for x in (q, k)]
        assert torch.equal(q_out, want[0]) and torch.equal(k_out, want[1])


def test_rows_past_32_bit_offsets():
    """Queries of 2.2e9 elements, in place: the last tokens' rows are turned, as their copies are."""
    n, d = 540_000, 128
    shape = kvc.make_shape(1, 1, 32, 32, d, 1)
    q = torch.zeros(1, 1, 32, n, d, dtype=torch.bfloat16, device="cuda")
    tail = make(1, 1, 32, 100, d, False, 1)
    q[:, :, :, -100:] = tail
    cos, sin = tables(1000, d)
    pos = (torch.arange(n, device="cuda") % 1000).to(torch.int32)[None]
    kvc.kvc_rope(shape, q, None, pos, cos, sin)
    assert torch.equal(q[:, :, :, -100:], rotated(tail, pos[:, -100:], cos, sin, HALF, d, False))
