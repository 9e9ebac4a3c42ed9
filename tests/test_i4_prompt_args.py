"""kvc_prompt_attn and the kvc_i4 calls refuse what they cannot do before they look for a device (CPU)."""
import ctypes
import os
import re

import pytest
import torch

import budgeted_kv_cache_gb300 as kvc

A = 1 << 20                                       # a 16-byte aligned stand-in pointer
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from budgeted_kv_cache_gb300 import build
    build.build()
    return kvc.library()


def shape(B=2, L=1, Hq=4, Hkv=2, d=64, T=100):
    return ctypes.byref(kvc.make_shape(B, L, Hq, Hkv, d, T))


def st(*v):
    return ctypes.byref(kvc.kvc_strides(*v))


def test_prompt_attention(lib):
    def call(sh=None, q=A, qs=None, n_q=8, k=A, v=A, ks=None, mods=None, out=A, os=None):
        return lib.kvc_prompt_attn(sh or shape(), q, qs, n_q, k, v, ks, None, None, None,
                                   ctypes.byref(mods) if mods else None, 0.0, out, os, None, None, None, 0, None)
    assert lib.kvc_prompt_attn(None, A, None, 8, A, A, None, None, None, None, None, 0.0, A, None, None, None, None, 0,
                               None) == INVALID
    assert call(sh=shape(d=96)) == UNSUPPORTED and call(sh=shape(Hq=3)) == INVALID
    assert call(n_q=0) == INVALID and call(n_q=-1) == INVALID
    assert call(sh=shape(Hq=64, Hkv=1), n_q=1 << 25) == UNSUPPORTED
    for bad in ("q", "k", "v", "out"):
        assert call(**{bad: None}) == INVALID and call(**{bad: A + 8}) == INVALID
    for bad in ("qs", "ks", "os"):
        assert call(**{bad: st(800, 0, 801, 64)}) == INVALID       # heads not 16-byte aligned
        assert call(**{bad: st(0, 0, 6400, 64)}) == INVALID        # a broadcast batch
        assert call(**{bad: st(1 << 20, 0, 6400, -64)}) == INVALID
    for bad in (kvc.kvc_score_mods(-1.0, None, 0, None), kvc.kvc_score_mods(float("nan"), None, 0, None),
                kvc.kvc_score_mods(float("inf"), None, 0, None), kvc.kvc_score_mods(0.0, None, -1, None)):
        assert call(mods=bad) == INVALID
    assert lib.kvc_prompt_attn_workspace_bytes(None, 4, 0) == 0
    assert lib.kvc_prompt_attn_workspace_bytes(shape(), 0, 0) == 0


def rows(**kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, pos=A, mass=A, count=A, next_pos=A, capacity=50, quant_mode=0)
    return ctypes.byref(kvc.kvc_i4_rows(*dict(f, **kw).values()))


BAD_ROWS = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(pos=None), dict(count=None),
            dict(next_pos=None), dict(k=A + 8), dict(v=A + 4), dict(k_scale=A + 2), dict(v_scale=A + 8),
            dict(capacity=0), dict(quant_mode=2)]


@pytest.mark.parametrize("bad", BAD_ROWS, ids=lambda b: "_".join(b))
def test_rows_of_a_4_bit_cache(lib, bad):
    r = rows(**bad)
    assert lib.kvc_i4_append(shape(), r, A, A, None, 1, None, None, None) == INVALID
    assert lib.kvc_i4_read(shape(), r, 1, A, A, None, None) == INVALID
    assert lib.kvc_i4_attn(shape(), r, A, None, 1, None, None, 0.0, 0, A, None, None, None, 0, None) == INVALID
    assert lib.kvc_i4_evict(shape(), r, 10, 0, 0, None, None, 0, None) == INVALID
    assert lib.kvc_i4_attn_workspace_bytes(shape(), r, 1, 1) == 0
    assert lib.kvc_i4_evict_workspace_bytes(shape(), r, 10) == 0


def test_4_bit_cache_calls(lib):
    append = lambda k=A, v=A, s=None, n=4, sh=None: lib.kvc_i4_append(sh or shape(), rows(), k, v, s, n, None, None, None)
    assert append(k=None) == INVALID and append(v=A + 2) == INVALID and append(n=-1) == INVALID
    assert append(s=st(0, 0, 256, 64)) == INVALID and append(s=st(512, 0, 256, 60)) == INVALID
    assert append(sh=shape(d=32)) == UNSUPPORTED
    assert append(n=0, k=None, v=None) == 0                     # nothing to append
    read = lambda n=4, k=A, v=A, s=None: lib.kvc_i4_read(shape(), rows(), n, k, v, s, None)
    assert read(n=51) == INVALID and read(n=-1) == INVALID and read(k=None) == INVALID and read(v=A + 8) == INVALID
    assert read(n=0, k=None, v=None) == 0
    attn = lambda r=None, q=A, n_q=1, fl=0, out=A, sh=None: lib.kvc_i4_attn(
        sh or shape(), r or rows(), q, None, n_q, None, None, 0.0, fl, out, None, None, None, 0, None)
    assert attn(q=None) == INVALID and attn(out=A + 8) == INVALID and attn(n_q=0) == INVALID
    assert attn(fl=2) == INVALID and attn(fl=1, r=rows(mass=None)) == INVALID
    assert attn(sh=shape(Hq=64, Hkv=1), n_q=1 << 25) == UNSUPPORTED
    evict = lambda b=10, s=0, n=0, r=None: lib.kvc_i4_evict(shape(), r or rows(), b, s, n, None, None, 0, None)
    assert evict(b=0) == INVALID and evict(s=-1) == INVALID and evict(n=-1) == INVALID and evict(r=rows(mass=None)) == INVALID


def test_binding_checks_tensors():
    """Wrong types, shapes and memory raise before the library is called."""
    s = kvc.make_shape(1, 1, 2, 2, 64, 8)
    x = torch.zeros(1, 1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(kvc.KvcError):                            # host memory
        kvc.kvc_prompt_attn(s, x, x, x, x.clone())
    ok = dict(k=torch.zeros(2, 8, 32, dtype=torch.uint8), v=torch.zeros(2, 8, 32, dtype=torch.uint8),
              k_scale=torch.zeros(2, 8, 2, dtype=torch.bfloat16), v_scale=torch.zeros(2, 8, 2, dtype=torch.bfloat16),
              pos=torch.zeros(2, 8, dtype=torch.int32), count=torch.zeros(2, dtype=torch.int32),
              next_pos=torch.zeros(2, dtype=torch.int32), mass=torch.zeros(2, 8))
    r = kvc.I4Rows(**ok)
    with pytest.raises(kvc.KvcError):
        kvc.kvc_i4_append(s, r, x, x)
    for bad in (dict(pos=torch.zeros(2, 8)), dict(k=torch.zeros(2, 8, 16, dtype=torch.uint8)),
                dict(k_scale=torch.zeros(2, 8, 2, dtype=torch.float16)), dict(count=torch.zeros(3, dtype=torch.int32)),
                dict(mass=torch.zeros(8, 2).T), dict(quant_mode=kvc.QUANT_ROW_FP16)):
        with pytest.raises(kvc.KvcError):
            kvc.I4Rows(**dict(ok, **bad))


def test_kernels_that_begin_early_load_coherently():
    """A kernel that may begin while the one before it still writes uses no load that is defined for data nobody writes
    during the kernel (read-only or non-coherent loads)."""
    csrc = os.path.join(os.path.dirname(os.path.abspath(kvc.__file__)), "csrc")
    sources = {f: open(os.path.join(csrc, f)).read() for f in os.listdir(csrc)}
    early = [f for f, text in sources.items() if f.endswith(".cu") and "launch_after(" in text]
    assert len(early) >= 3
    for f in early + ["packed_math.cuh"]:
        code = re.sub(r"//.*", "", sources[f])
        assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", code), f


def test_slot_numbers_stay_within_31_bits(lib):
    """Capacities and appends so near 2^31 that a block's step past the last row would leave 31 bits are refused."""
    most = 0x7fff0000
    assert lib.kvc_i4_append(shape(), rows(), A, A, None, most + 1, None, None, None) == UNSUPPORTED
    for capacity in (most + 1, 2 ** 31 - 1):
        r = rows(capacity=capacity)
        assert lib.kvc_i4_append(shape(), r, A, A, None, 1, None, None, None) == UNSUPPORTED
        assert lib.kvc_i4_read(shape(), r, 1, A, A, None, None) == UNSUPPORTED
        assert lib.kvc_i4_attn(shape(), r, A, None, 1, None, None, 0.0, 1, A, None, None, None, 0, None) == UNSUPPORTED
        assert lib.kvc_i4_evict(shape(), r, 10, 0, 0, None, None, 0, None) == UNSUPPORTED
        assert lib.kvc_i4_evict_workspace_bytes(shape(), r, 10) == 0
    # the largest that is allowed: every index that the kernels form (per unit) fits
    step = 16384 + 8 * 1024
    assert most + step < 2 ** 31 and kvc.library().kvc_i4_evict_workspace_bytes(shape(), rows(capacity=most), 10) > 0
