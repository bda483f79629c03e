"""The table of frequencies against its formula in 60 decimal digits, and its refusals.  Host only."""
import math
from decimal import Decimal, getcontext

import pytest

from replicated_fp8_sparse_amd import kvpub

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
TAU = 2 * PI


def power(base, exponent):
    return (Decimal(base).ln() * Decimal(exponent)).exp()


def want(dim, scaling, base, factor, original, low, high):
    base, factor, original, low, high = (Decimal(v) for v in (base, factor, original, low, high))
    if scaling == kvpub.SCALING_GROWN:
        base *= power(factor, Decimal(dim) / Decimal(dim - 2))
    at = lambda t: Decimal(dim) * (original / (TAU * t)).ln() / (2 * base.ln())
    out = []
    for i in range(dim // 2):
        f = power(base, Decimal(-2 * i) / Decimal(dim))
        keep = Decimal(1)
        if scaling == kvpub.SCALING_LINEAR:
            keep = Decimal(0)
        if scaling == kvpub.SCALING_RAMP:
            lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), dim - 1)
            keep = 1 - min(max((i - Decimal(lo)) / max(Decimal(hi - lo), Decimal("0.001")), Decimal(0)), Decimal(1))
        if scaling == kvpub.SCALING_BLEND:
            keep = min(max((original * f / TAU - low) / (high - low), Decimal(0)), Decimal(1))
        out.append((f * keep + f / factor * (1 - keep)) / TAU * 2 ** 64)
    return out


@pytest.mark.parametrize("scaling", range(5))
@pytest.mark.parametrize("dim,base,factor,original", [(8, 10000.0, 4.0, 2048.0), (64, 10000.0, 40.0, 4096.0), (48, 500000.0, 8.0, 8192.0),
                                                      (128, 1000000.0, 1.0, 32768.0), (1024, 1.5, 3.7, 100.0)])
def test_turns(dim, base, factor, original, scaling):
    low, high = 1.0, 32.0
    st, got = kvpub.kvpub_rotation_turns(kvpub.rotation_config(dim, base, scaling, factor, original, low, high))
    assert st == kvpub.KVPUB_OK and len(got) == dim // 2
    for i, (g, w) in enumerate(zip(got, want(dim, scaling, base, factor, original, low, high))):
        # 64-bit significands: the exponent's rounding times ln(base) (below 14), the power's own, a few products: 2^-59
        # of the value at most, and the last rounding to a whole number.  RAMP's and BLEND's weights multiply a difference
        # of order 1: 2^-59 of f again.
        assert abs(Decimal(int(g)) - w) <= w * Decimal(2) ** -58 + Decimal(2) ** 64 / TAU * Decimal(2) ** -60 * (scaling >= 3) + 1, i


def test_first_pair_turns_one_radian():
    _, got = kvpub.kvpub_rotation_turns(kvpub.rotation_config(64))
    # 2^64 / tau is below 2^61.4; tau rounded to 64 bits and the division are off by 2^-64 of it each, which is
    # 0.34 in all, and the last rounding by 0.5: below 1
    assert abs(int(got[0]) - Decimal(2) ** 64 / TAU) < 1


@pytest.mark.parametrize("change", [dict(dim=0), dict(dim=12), dict(dim=1032), dict(scaling=5), dict(base=1.0), dict(base=-3.0),
                                    dict(base=math.inf), dict(base=math.nan), dict(scaling=1, factor=0.5),
                                    dict(scaling=1, factor=math.nan), dict(scaling=3, original=0.0), dict(scaling=3, original=math.inf),
                                    dict(scaling=4, low=0.0), dict(scaling=4, low=math.nan), dict(scaling=4, low=5.0, high=5.0),
                                    dict(scaling=3, high=math.inf), dict(scaling=3, high=math.nan)])
def test_refusals(change):
    c = kvpub.rotation_config(64, factor=2.0, original=100.0, low=1.0, high=32.0)
    for k, v in change.items():
        setattr(c, k, v)
    assert kvpub.kvpub_rotation_turns(c) == (kvpub.KVPUB_ERR_INVALID_ARG, None)


def test_what_a_scaling_does_not_read_is_not_checked():
    c = kvpub.rotation_config(64, scaling=kvpub.SCALING_NONE, factor=math.nan, original=-1.0, low=-1.0, high=-2.0)
    assert kvpub.kvpub_rotation_turns(c)[0] == kvpub.KVPUB_OK
    c = kvpub.rotation_config(64, scaling=kvpub.SCALING_GROWN, factor=4.0, original=-1.0, low=-1.0, high=-2.0)
    assert kvpub.kvpub_rotation_turns(c)[0] == kvpub.KVPUB_OK
    assert kvpub.load().kvpub_rotation_turns(None, None) == kvpub.KVPUB_ERR_INVALID_ARG
