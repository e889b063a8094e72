"""Frequency tables of rotary positions against 60-digit arithmetic: every entry is the frequency in turns, modulo one
turn, rounded to 2^-64 (one unit of it: half for the rounding, the rest for values near the middle of two)."""
import decimal
import os

import pytest

import overlapped_tensor_gemm_gb300 as fo

D = decimal.Decimal
TWO_PI = 2 * D("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(fo.LIB_PATH):
        from overlapped_tensor_gemm_gb300 import _build
        _build.build()
    return fo.load()


def _turns(rot, base, scaling=None, factor=1.0, low=1.0, high=4.0, length=0, first=0, last=0):
    out = []
    with decimal.localcontext() as c:
        c.prec = 60
        for i in range(rot // 2):
            f = (D(-2 * i) / rot * D(base).ln()).exp()
            keep = D(1)
            if scaling == "linear":
                keep = D(0)
            elif scaling == "banded":
                keep = (D(length) * f / TWO_PI - D(low)) / (D(high) - D(low))
            elif scaling == "ramped":
                keep = 1 - D(i - first) / (last - first)
            keep = min(max(keep, D(0)), D(1))
            out.append(((1 - keep) * f / D(factor) + keep * f) / TWO_PI)
    return out


def _check(table, want):
    with decimal.localcontext() as c:
        c.prec = 60
        for i, w in enumerate(want):
            off = (D(table.c.turns[i]) - w * 2 ** 64) % 2 ** 64
            off = min(off, 2 ** 64 - off)
            assert off <= 1, (i, table.c.turns[i], float(off))


@pytest.mark.parametrize("rot,base", [(128, 10000.0), (64, 500000.0), (2, 10000.0), (512, 100.0), (96, 1.5), (256, 1e7),
                                      (32, 1e300)])
@pytest.mark.parametrize("kw", [{}, dict(scaling="linear", factor=4.0), dict(scaling="linear", factor=0.05),
                                dict(scaling="banded", factor=8.0, length=8192)], ids=str)
def test_turns(rot, base, kw):
    how = {("original_length" if k == "length" else k): v for k, v in kw.items()}
    _check(fo.RopeTable(rot, base=base, **how), _turns(rot, base, **kw))


def test_ramped_turns():
    # 128 dimensions, base 10000, 4096 positions: 32 turns at pair 20.9.., 1 turn at pair 45.0..
    with decimal.localcontext() as c:
        c.prec = 60
        pair = lambda t: 128 * (D(4096) / (TWO_PI * t)).ln() / (2 * D(10000).ln())  # noqa: E731
        first, last = int(pair(32).to_integral_value(decimal.ROUND_FLOOR)), int(pair(1).to_integral_value(decimal.ROUND_CEILING))
    _check(fo.RopeTable(128, scaling="ramped", factor=16.0, original_length=4096),
           _turns(128, 10000.0, scaling="ramped", factor=16.0, first=first, last=last))
