"""The angles of kvc_rope_tables against 80 decimal digits, at positions up to 2^31 - 1 (CPU: the host's part, compiled alone)."""
import ctypes
import math
import os
import shutil
import subprocess
from decimal import Decimal, getcontext

import pytest

import budgeted_kv_cache_gb300 as kvc

getcontext().prec = 80
TAU = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """#include "rope_turns.h"
extern "C" int turns(int rot, double base, const kvc_rope_scaling* s, uint64_t* to, float* magnitude) {
  return kvc::rope_turns(rot, base, s, to, magnitude);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no host compiler")
    where = tmp_path_factory.mktemp("turns")
    (where / "turns.cpp").write_text(CODE)
    csrc = os.path.join(ROOT, "budgeted_kv_cache_gb300", "csrc")
    r = subprocess.run([gxx, "-O3", "-std=c++17", "-shared", "-fPIC", "-I", csrc, "-I", os.path.join(ROOT, "include"),
                        str(where / "turns.cpp"), "-o", str(where / "turns.so")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    so = ctypes.CDLL(str(where / "turns.so"))
    so.turns.argtypes = [ctypes.c_int, ctypes.c_double, ctypes.POINTER(kvc.kvc_rope_scaling), ctypes.c_void_p, ctypes.c_void_p]
    return so


def exact(rot, base, s):
    """Turns per position, from the header's definition."""
    base, f, half = Decimal(base), Decimal(s.factor), rot // 2
    if s.kind == kvc.ROPE_SCALE_BASE:
        base *= f ** (Decimal(rot) / (rot - 2))
    out = []
    for i in range(half):
        theta, keep = base ** (Decimal(-2 * i) / rot), Decimal(1)
        if s.kind == kvc.ROPE_SCALE_LINEAR:
            keep = Decimal(0)
        elif s.kind == kvc.ROPE_SCALE_TURNS:
            keep = (Decimal(s.original_len) * theta / TAU - Decimal(s.low)) / (Decimal(s.high) - Decimal(s.low))
        elif s.kind == kvc.ROPE_SCALE_DIMS:
            at = lambda n: rot * math.log(s.original_len / (2 * math.pi * n)) / (2 * math.log(float(base)))
            a, b = max(math.floor(at(s.high)), 0), min(math.ceil(at(s.low)), rot - 1)
            keep = 1 - Decimal(i - a) / Decimal(max(float(b - a), 0.001))
        keep = min(max(keep, Decimal(0)), Decimal(1))
        out.append(theta / TAU * (keep + (1 - keep) / f))
    return out


SCALINGS = [kvc.RopeScaling(), kvc.RopeScaling(kvc.ROPE_SCALE_LINEAR, 8.0), kvc.RopeScaling(kvc.ROPE_SCALE_LINEAR, 3.7),
            kvc.RopeScaling(kvc.ROPE_SCALE_LINEAR, 0.05), kvc.RopeScaling(kvc.ROPE_SCALE_LINEAR, 1e-3),
            kvc.RopeScaling(kvc.ROPE_SCALE_BASE, 4.3), kvc.RopeScaling(kvc.ROPE_SCALE_BASE, 0.7),
            kvc.RopeScaling(kvc.ROPE_SCALE_TURNS, 32.0, 8192.0, 1.0, 4.0), kvc.RopeScaling(kvc.ROPE_SCALE_TURNS, 40.3, 2048.0, 0.0, 0.5),
            kvc.RopeScaling(kvc.ROPE_SCALE_DIMS, 16.0, 4096.0, 1.0, 32.0), kvc.RopeScaling(kvc.ROPE_SCALE_DIMS, 7.3, 32768.0, 0.9, 33.0)]


@pytest.mark.parametrize("s", SCALINGS, ids=range(len(SCALINGS)))
@pytest.mark.parametrize("rot", [16, 48, 112, 128])
@pytest.mark.parametrize("base", [1e4, 5e5, 1e6, 1.5, 12345.678, 1e30])
def test_turns(lib, base, rot, s):
    to = (ctypes.c_uint64 * 64)()
    magnitude = ctypes.c_float()
    c = kvc.kvc_rope_scaling(s.kind, s.factor, s.original_len, s.low, s.high, s.magnitude)
    valid = s.kind != kvc.ROPE_SCALE_BASE or base * s.factor ** (rot / (rot - 2)) >= 1      # a scaled base below 1 is refused
    assert lib.turns(rot, base, ctypes.byref(c), to, ctypes.byref(magnitude)) == valid
    if not valid:
        return
    assert magnitude.value == s.magnitude
    for i, want in enumerate(exact(rot, base, s)):
        off = (to[i] - int((want % 1) * 2 ** 64)) % 2 ** 64
        # half a unit from each double of the sum, and the whole number wanted is rounded down
        assert min(off, 2 ** 64 - off) <= 2, (i, off)
        for p in (1, 131071, 50_000_000, 2 ** 31 - 1):
            turn, angle = Decimal(to[i] * p % 2 ** 64) / 2 ** 64, want * p % 1
            apart = abs(turn - angle)
            # half a unit from each double of the sum: p 2^-64 turns, 2^-30 of angle at most, where the tables' 2^-22 leaves
            # 1.3e-7 = 2^-23 beside their polynomials' 1e-7
            assert min(apart, 1 - apart) <= Decimal(p) * Decimal("1.01") / 2 ** 64, (i, p)


def test_without_a_scaling(lib):
    to, magnitude = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    assert lib.turns(64, 10000.0, None, to, ctypes.byref(magnitude)) == 1 and magnitude.value == 1.0
    assert to[0] == round(2 ** 64 / TAU) and not lib.turns(64, 0.5, None, to, ctypes.byref(magnitude))
