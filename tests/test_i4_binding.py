"""Tensors that the binding of the prompt attention and the 4-bit cache takes and refuses (CPU: helpers with the host's
device number, -1; GPU: the calls)."""
import pytest
import torch

import budgeted_kv_cache_gb300 as kvc


def bf16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def views(make):
    """Keys and values of one sequence and layer that lie alike but for the strides of the dimensions of size 1."""
    k = make(3, 1, 4, 20, 64)[1:2, :, :, :8]                   # one sequence of three
    v = make(1, 2, 4, 20, 64)[:, 1:2, :, :8]                   # one layer of two
    return k, v


def test_strides_of_single_dimensions_are_not_compared():
    s = kvc.make_shape(1, 1, 8, 4, 64, 8)
    k, v = views(bf16)
    assert k.stride() != v.stride()
    assert kvc._pair("f", -1, k, v, s, 8) is not None
    assert kvc._pair("f", -1, v, k, s, 8) is not None
    for other in (bf16(1, 1, 4, 8, 64), bf16(1, 1, 4, 21, 64)[:, :, :, :8], bf16(1, 1, 20, 4, 64).transpose(2, 3)[:, :, :, :8]):
        for pair in ((k, other), (other, k)):
            with pytest.raises(kvc.KvcError):
                kvc._pair("f", -1, *pair, s, 8)


def rows_on_the_host():
    s = kvc.make_shape(1, 1, 2, 2, 64, 1)
    return s, kvc.I4Rows.allocate(s, 8, device="cpu")


def test_replaced_tensors_of_a_cache_are_checked():
    """What takes a tensor's place later has to fit as well: kernels index it by the codes' capacity."""
    i32 = torch.int32
    for name, bad in (("mass", torch.zeros(2, 7)), ("mass", torch.zeros(2, 8, dtype=torch.float64)),
                      ("pos", torch.zeros(2, 9, dtype=i32)), ("count", torch.zeros(1, dtype=i32)),
                      ("next_pos", torch.zeros(2, dtype=torch.int64)), ("v", torch.zeros(2, 8, 16, dtype=torch.uint8)),
                      ("k_scale", torch.zeros(2, 8, 1, dtype=torch.bfloat16)), ("quant_mode", kvc.QUANT_ROW_FP16),
                      ("pos", torch.zeros(8, 2, dtype=i32).T)):
        s, rows = rows_on_the_host()
        kvc._cache("f", -1, rows, s)
        setattr(rows, name, bad)
        for _ in range(2):                                     # still refused the second time
            with pytest.raises(kvc.KvcError):
                kvc._cache("f", -1, rows, s)
    # one that fits, none, and all of them in turn for a larger cache
    s, rows = rows_on_the_host()
    for mass in (torch.zeros(2, 8), None):
        rows.mass = mass
        kvc._cache("f", -1, rows, s)
    larger = kvc.I4Rows.allocate(s, 16, device="cpu")
    for name in ("k", "v", "k_scale", "v_scale", "pos", "mass", "count", "next_pos"):
        setattr(rows, name, getattr(larger, name))
    kvc._cache("f", -1, rows, s)
    assert rows.c().capacity == 16


def test_numbers_that_the_c_types_would_change_are_refused():
    """2^32 + 5 as a window of 5, 2^32 recent rows as none, a cap of 1e-50 as no cap."""
    s, rows = rows_on_the_host()
    for mods in (kvc.ScoreMods(window=2 ** 32 + 5), kvc.ScoreMods(window=2 ** 31), kvc.ScoreMods(softcap=1e-50)):
        with pytest.raises(kvc.KvcError):
            kvc._mods("f", -1, mods, s)
    for mods in (kvc.ScoreMods(window=2 ** 31 - 1), kvc.ScoreMods(softcap=1e-42), kvc.ScoreMods(softcap=0.0)):
        assert kvc._mods("f", -1, mods, s) is not None
    with pytest.raises(kvc.KvcError):
        kvc.kvc_prompt_attn_workspace_bytes(s, 2 ** 32 + 1)
    with pytest.raises(kvc.KvcError):
        kvc.kvc_i4_attn_workspace_bytes(s, rows, 2 ** 32 + 1)
    with pytest.raises(kvc.KvcError):
        kvc.kvc_i4_evict_workspace_bytes(s, rows, 2 ** 32 + 1)


@pytest.mark.gpu
def test_eviction_numbers_past_32_bits_are_refused():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s = kvc.make_shape(1, 1, 2, 2, 64, 1)
    rows = kvc.I4Rows.allocate(s, 8)
    x = torch.randn(1, 1, 2, 8, 64, device="cuda").to(torch.bfloat16)
    kvc.kvc_i4_append(s, rows, x, x)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    for bad in ((2 ** 32 + 4, 0, 0), (4, 2 ** 32, 0), (4, 0, 2 ** 32)):
        with pytest.raises(kvc.KvcError):
            kvc.kvc_i4_evict(s, rows, *bad, workspace=ws)
    assert rows.count.tolist() == [8, 8]


@pytest.mark.gpu
def test_calls_with_views_that_differ_in_single_dimensions():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from budgeted_kv_cache_gb300 import build
    build.build()
    make = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)
    s = kvc.make_shape(1, 1, 8, 4, 64, 8)
    k, v = views(make)
    q, got, want = make(1, 1, 8, 8, 64), bf16(1, 1, 8, 8, 64).cuda(), bf16(1, 1, 8, 8, 64).cuda()
    ws = torch.empty(max(256, kvc.kvc_prompt_attn_workspace_bytes(s, 8)), dtype=torch.uint8, device="cuda")
    kvc.kvc_prompt_attn(s, q, k, v, got, workspace=ws)
    kvc.kvc_prompt_attn(s, q, k.contiguous(), v.contiguous(), want, workspace=ws)
    assert torch.equal(got, want)
    rows = [kvc.I4Rows.allocate(s, 8) for _ in range(2)]
    kvc.kvc_i4_append(s, rows[0], k, v)
    kvc.kvc_i4_append(s, rows[1], k.contiguous(), v.contiguous())
    assert torch.equal(rows[0].k, rows[1].k) and torch.equal(rows[0].v, rows[1].v)
    outs = [views(make), (bf16(1, 1, 4, 8, 64).cuda(), bf16(1, 1, 4, 8, 64).cuda())]
    for o in outs:
        kvc.kvc_i4_read(s, rows[0], *o)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
