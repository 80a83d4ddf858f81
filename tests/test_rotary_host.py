"""Refusals of h2o_rotate that reach no device, and the binding's fractions of a turn (CPU)."""
from __future__ import annotations

import ctypes as C
import math
from fractions import Fraction

import pytest

import h2o_heavy_hitter_decode_gb300 as h2o
from h2o_heavy_hitter_decode_gb300 import build as hbuild
from h2o_heavy_hitter_decode_gb300.rotary import TWO_PI, _Rotary

F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    hbuild.build()
    return h2o.lib()


def call(L, desc=None, dtype=BF16, B=2, n=3, hq=4, hk=2, q=None, k=None, position=256, counts=None, qo=None, ko=None, **over):
    fields = dict(d=64, pairs=32, interleaved=0, axes=1, norm=1, eps=1e-6, turns=256, axis=256, q_weight=256, k_weight=256)
    fields.update(over)
    good = (4096, 4 * 3 * 64, 3 * 64, 64)
    rows = [C.byref(h2o.Rows(*(x or good))) if x is not False else None for x in (q, k, qo, ko)]
    d = None if desc is False else C.byref(_Rotary(*fields.values()))
    return L.h2o_rotate(d, dtype, B, n, hq, hk, rows[0], rows[1], position, 0, counts, rows[2], rows[3], None)


@pytest.mark.parametrize("bad", [
    dict(desc=False), dict(dtype=2), dict(dtype=-1), dict(d=0), dict(pairs=-8), dict(pairs=12), dict(pairs=40), dict(axes=0),
    dict(eps=-1.0), dict(eps=math.nan), dict(turns=None), dict(turns=260), dict(q_weight=264), dict(k_weight=264),
    dict(position=None), dict(position=258), dict(counts=258), dict(B=0), dict(n=0), dict(hq=-1), dict(hq=0, hk=0),
    dict(hq=1 << 25), dict(B=1 << 16, n=1 << 16), dict(q=False), dict(k=False), dict(qo=False), dict(ko=False),
    dict(q=(4104, 768, 192, 64)), dict(k=(4096, 768, 192, 60)), dict(k=(4096, -768, 192, 64)),
    dict(qo=(4096, 768, 128, 64)), dict(qo=(4096, 768, 0, 64)), dict(dtype=F32, q=(4096, 768, 192, 66)),
], ids=str)
def test_refused(L, bad):
    assert call(L, **bad) == 1


def test_unsupported_head_size(L):
    assert call(L, d=96, pairs=48) == 6


def test_two_pi():
    assert abs(float(TWO_PI) - 2 * math.pi) == 0.0
    # Machin: pi = 16 atan(1/5) - 4 atan(1/239), to 60 digits
    def atan_inverse(x):
        total, term, k = Fraction(0), Fraction(1, x), 0
        while term > Fraction(1, 10 ** 60):
            total += (-1) ** k * term / (2 * k + 1)
            term, k = term / x ** 2, k + 1
        return total
    pi = 16 * atan_inverse(5) - 4 * atan_inverse(239)
    assert abs(TWO_PI - 2 * pi) < Fraction(1, 10 ** 48)


def test_binding_refuses_before_the_device():
    for bad in (dict(d=96), dict(d=64, dims=24), dict(d=64, eps=-1.0), dict(d=64, device="cpu")):
        with pytest.raises(ValueError):
            h2o.H2ORotary(**bad)
