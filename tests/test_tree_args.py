"""kvc_i4_tree_attn and kvc_i4_tree_commit refuse what they cannot do before they look for a device (CPU)."""
import ctypes

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


def rows(**kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, pos=A, mass=A, count=A, next_pos=A, capacity=50, quant_mode=0)
    return ctypes.byref(kvc.kvc_i4_rows(*dict(f, **kw).values()))


BAD_ROWS = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(pos=None), dict(count=None),
            dict(next_pos=None), dict(k=A + 8), dict(v=A + 4), dict(k_scale=A + 2), dict(v_scale=A + 8),
            dict(capacity=0), dict(quant_mode=2)]


def attn(lib, sh=None, r=None, q=A, qs=None, n=8, k=A, v=A, ks=None, parent=A, mods=None, out=A, os=None):
    return lib.kvc_i4_tree_attn(sh or shape(), r or rows(), q, qs, n, k, v, ks, parent, None,
                                ctypes.byref(mods) if mods else None, 0.0, out, os, None, None, None, 0, None)


@pytest.mark.parametrize("bad", BAD_ROWS, ids=lambda b: "_".join(b))
def test_rows_of_a_4_bit_cache(lib, bad):
    assert attn(lib, r=rows(**bad)) == INVALID
    assert lib.kvc_i4_tree_attn_workspace_bytes(shape(), rows(**bad), 4) == 0


def test_attention(lib):
    assert attn(lib, sh=shape(d=96)) == UNSUPPORTED and attn(lib, sh=shape(Hq=3)) == INVALID
    assert attn(lib, n=0) == INVALID and attn(lib, n=-1) == INVALID
    assert attn(lib, n=kvc.TREE_MAX_NODES + 1) == UNSUPPORTED
    assert attn(lib, r=rows(capacity=0x7fff0001)) == UNSUPPORTED
    for bad in ("q", "k", "v", "out"):
        assert attn(lib, **{bad: None}) == INVALID and attn(lib, **{bad: A + 8}) == INVALID
    assert attn(lib, parent=None) == INVALID
    for bad in ("qs", "ks", "os"):
        assert attn(lib, **{bad: st(800, 0, 801, 64)}) == INVALID       # heads not 16-byte aligned
        assert attn(lib, **{bad: st(0, 0, 6400, 64)}) == INVALID        # a broadcast batch
        assert attn(lib, **{bad: st(1 << 20, 0, 6400, -64)}) == INVALID
    for bad in (kvc.kvc_score_mods(-1.0, None, 0, None), kvc.kvc_score_mods(float("nan"), None, 0, None),
                kvc.kvc_score_mods(float("inf"), None, 0, None), kvc.kvc_score_mods(0.0, None, -1, None)):
        assert attn(lib, mods=bad) == INVALID
    assert lib.kvc_i4_tree_attn_workspace_bytes(None, rows(), 4) == 0
    assert lib.kvc_i4_tree_attn_workspace_bytes(shape(), rows(), 0) == 0
    assert lib.kvc_i4_tree_attn_workspace_bytes(shape(), rows(), kvc.TREE_MAX_NODES + 1) == 0


def commit(lib, sh=None, r=None, k=A, v=A, ks=None, n=8, path=A, size=A, steps=4, q=A, qs=None, lse=A, mods=None, ko=A + 4096,
           vo=A + 8192, os=None):
    return lib.kvc_i4_tree_commit(sh or shape(), r or rows(), k, v, ks, n, path, size, steps, q, qs, lse,
                                  ctypes.byref(mods) if mods else None, 0.0, ko, vo, os, None, None)


@pytest.mark.parametrize("bad", BAD_ROWS, ids=lambda b: "_".join(b))
def test_rows_of_a_commit(lib, bad):
    assert commit(lib, r=rows(**bad)) == INVALID


def test_commit(lib):
    assert commit(lib, sh=shape(d=96)) == UNSUPPORTED and commit(lib, sh=shape(Hq=3)) == INVALID
    assert commit(lib, n=0) == INVALID and commit(lib, n=kvc.TREE_MAX_NODES + 1) == UNSUPPORTED
    assert commit(lib, steps=0) == INVALID and commit(lib, steps=9) == INVALID and commit(lib, steps=-1) == INVALID
    assert commit(lib, n=100, steps=kvc.TREE_MAX_PATH + 1) == UNSUPPORTED
    assert commit(lib, r=rows(capacity=0x7fff0001)) == UNSUPPORTED
    for bad in ("k", "v", "path", "size", "lse", "ko", "vo"):
        assert commit(lib, **{bad: None}) == INVALID
    for bad in ("k", "v", "q", "ko", "vo"):
        assert commit(lib, **{bad: A + 8}) == INVALID
    assert commit(lib, ko=A) == INVALID and commit(lib, vo=A) == INVALID and commit(lib, ko=A + 4096, vo=A + 4096) == INVALID
    assert commit(lib, v=A + 4096) == INVALID and commit(lib) not in (INVALID, UNSUPPORTED)
    assert commit(lib, r=rows(mass=None)) == INVALID             # weights with nowhere to go
    for bad in ("ks", "qs", "os"):
        assert commit(lib, **{bad: st(800, 0, 801, 64)}) == INVALID
        assert commit(lib, **{bad: st(0, 0, 6400, 64)}) == INVALID
    for bad in (kvc.kvc_score_mods(-1.0, None, 0, None), kvc.kvc_score_mods(0.0, None, -1, None)):
        assert commit(lib, mods=bad) == INVALID


def test_binding_refuses_tensors_on_the_host():
    s = kvc.make_shape(1, 1, 2, 2, 64, 1)
    x, parent = torch.zeros(1, 1, 2, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 8, dtype=torch.int32)
    r = kvc.I4Rows.allocate(s, 8, device="cpu")
    with pytest.raises(kvc.KvcError):
        kvc.kvc_i4_tree_attn(s, r, x, x, x, parent, x.clone())
    with pytest.raises(kvc.KvcError):
        kvc.kvc_i4_tree_attn_workspace_bytes(s, r, 2 ** 32 + 1)
    path, size = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(kvc.KvcError):
        kvc.kvc_i4_tree_commit(s, r, x, x, path, size)
