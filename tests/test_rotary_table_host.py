"""The rotary table against 60-digit arithmetic, and the angle that the kernel makes of it against the bound that the header
gives: 2^-24 of a half turn at any position (no GPU)."""
import decimal
import random

import numpy as np
import pytest

from sparse_attention_kpool_gb300 import build as kbuild
from sparse_attention_kpool_gb300 import kpool as K

D = decimal.Decimal
PI = D("3.14159265358979323846264338327950288419716939937510582097494459")
KINDS = [(128, {}), (2, {}), (64, dict(base=500000.0, factor=8.0, original_length=8192.0, high=4.0)), (96, dict(factor=4.0)),
         (64, dict(factor=40.0, original_length=4096.0)), (20, dict(base=1.5)), (256, dict(base=1e9)), (6, dict(base=0.25))]
FAR = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 3, 10 ** 9 + 7, 1 << 20, 131071, -(1 << 30) - 1]


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()


def turns(rd, base=10000.0, factor=1.0, original_length=0.0, low=1.0, high=32.0):
    """Turns a token of each pair, to 60 digits."""
    with decimal.localcontext(decimal.Context(prec=60)):
        b, fac, orig, lo, hi = (D(x) for x in (base, factor, original_length, low, high))
        out = []
        for i in range(rd // 2):
            f = (b.ln() * (D(-2 * i) / rd)).exp() / (2 * PI)
            keep = min(D(1), max(D(0), (orig * f - lo) / (hi - lo))) if orig else D(0)
            out.append(f * (keep + (1 - keep) / fac))
        return out


@pytest.mark.parametrize("rd,kw", KINDS, ids=str)
def test_table_to_its_last_places(rd, kw):
    """Sums, products and a power of 64 bits each are off by 5 steps of 2^-64 of the value at most, and as much again, times
    high / (high - low) <= 4 / 3, where a pair is stretched in part; below a turn (base >= 1: 0.16) that is two units of
    2^-64 and the rounding to whole ones. Bases below 1 turn faster."""
    table = K.new_rotary_table(rd, device="cpu", **kw).tolist()
    with decimal.localcontext(decimal.Context(prec=60)):
        for got, want in zip(table, turns(rd, **kw)):
            off = abs(got % 2 ** 64 - want % 1 * 2 ** 64)
            assert min(off, 2 ** 64 - off) <= 4 * max(1, want / D("0.16")), (got, want)


@pytest.mark.parametrize("rd,kw", KINDS, ids=str)
def test_angles_at_any_position(rd, kw):
    rng = random.Random(rd)
    positions = FAR + [rng.randrange(-2 ** 31, 2 ** 31) for _ in range(60)]
    table = K.new_rotary_table(rd, device="cpu", **kw).tolist()
    with decimal.localcontext(decimal.Context(prec=60)):
        for word, f in zip(table, turns(rd, **kw)):
            for t in positions:
                x = (t * word) % 2 ** 64
                top = np.int64(x >> 32).astype(np.int32)
                half_turns = D(float(np.float32(top))) / 2 ** 31
                off = (half_turns - 2 * t * f) % 2
                assert min(off, 2 - off) <= D(2) ** -24, (t, f)

