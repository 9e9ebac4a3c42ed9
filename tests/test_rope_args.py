"""kvc_rope_tables and kvc_rope refuse what they cannot do before they look for a device (CPU)."""
import ctypes
import math

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


def shape(B=2, L=1, Hq=4, Hkv=2, d=64, T=1):
    return ctypes.byref(kvc.make_shape(B, L, Hq, Hkv, d, T))


def st(*v):
    return ctypes.byref(kvc.kvc_strides(*v))


def scaled(**kw):
    f = dict(kind=kvc.ROPE_SCALE_TURNS, factor=4.0, original_len=4096.0, low=1.0, high=32.0, magnitude=1.0)
    return ctypes.byref(kvc.kvc_rope_scaling(*dict(f, **kw).values()))


BAD_SCALING = [dict(kind=-1), dict(kind=5), dict(factor=0.0), dict(factor=-1.0), dict(factor=math.inf), dict(factor=math.nan),
               dict(original_len=0.0), dict(original_len=math.inf), dict(original_len=math.nan), dict(low=-1.0), dict(low=math.nan),
               dict(low=32.0), dict(high=math.inf), dict(high=math.nan), dict(magnitude=math.inf), dict(magnitude=math.nan),
               dict(kind=kvc.ROPE_SCALE_DIMS, low=0.0), dict(kind=kvc.ROPE_SCALE_LINEAR, factor=0.0),
               dict(kind=kvc.ROPE_SCALE_BASE, factor=1e-9)]


@pytest.mark.parametrize("bad", BAD_SCALING, ids=lambda b: "_".join(f"{k}={v}" for k, v in b.items()))
def test_scalings(lib, bad):
    assert lib.kvc_rope_tables(8, 64, 10000.0, scaled(**bad), A, A, None) == INVALID


def test_tables(lib):
    call = lambda n=8, rot=64, base=1e4, s=None, c=A, x=A: lib.kvc_rope_tables(n, rot, base, s, c, x, None)
    for bad in (dict(n=-1), dict(n=1 << 31), dict(rot=0), dict(rot=24), dict(rot=144), dict(rot=-16), dict(base=0.5),
                dict(base=math.inf), dict(base=math.nan), dict(c=None), dict(x=None), dict(c=A + 4), dict(x=A + 8)):
        assert call(**bad) == INVALID, bad
    assert call(s=scaled(kind=kvc.ROPE_SCALE_DIMS), base=1.0) == INVALID
    assert call(n=0, c=None, x=None) == 0                        # nothing to fill


def test_rotation(lib):
    def call(sh=None, q=A, qs=None, k=A, ks=None, n=8, pos=A, cos=A, sin=A, top=100, layout=0, rot=0, flags=0, qo=A + 4096,
             qos=None, ko=A + 8192, kos=None):
        return lib.kvc_rope(sh or shape(), q, qs, k, ks, n, pos, None, cos, sin, top, layout, rot, flags, qo, qos, ko, kos, None,
                            None)
    assert call(sh=shape(Hq=3)) == INVALID and call(sh=shape(d=96)) == UNSUPPORTED
    for bad in (dict(n=-1), dict(rot=8), dict(rot=80), dict(rot=24), dict(rot=-16), dict(layout=2), dict(layout=-1), dict(flags=2),
                dict(top=0), dict(pos=None), dict(cos=None), dict(sin=None), dict(cos=A + 4), dict(q=None), dict(qo=None),
                dict(k=None), dict(ko=None), dict(q=A + 8), dict(k=A + 2), dict(qo=A + 8), dict(ko=A + 8),
                dict(qs=st(800, 0, 801, 64)), dict(ks=st(0, 0, 512, 64)), dict(qos=st(1 << 20, 0, 512, -64)),
                dict(kos=st(1 << 20, 0, 512, 60))):
        assert call(**bad) == INVALID, bad
    assert call(qo=A, qs=st(4096, 0, 1024, 64)) == INVALID       # in place with other strides
    assert call(ko=A, kos=st(4096, 0, 64, 128)) == INVALID
    assert call(n=0, pos=None, cos=None) == 0 and call(q=None, qo=None, k=None, ko=None, pos=None) == 0
    assert lib.kvc_rope(None, A, None, A, None, 8, A, None, A, A, 8, 0, 0, 0, A, None, A, None, None, None) == INVALID


def test_binding_refuses_tensors_on_the_host():
    s = kvc.make_shape(1, 1, 2, 2, 64, 1)
    x, pos, t = torch.zeros(1, 1, 2, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 8, dtype=torch.int32), torch.zeros(9, 32)
    with pytest.raises(kvc.KvcError):
        kvc.kvc_rope(s, x, x.clone(), pos, t, t.clone())
    with pytest.raises(kvc.KvcError):
        kvc.kvc_rope_tables(t, t.clone())
