"""Speculative decoding without a GPU, where it can go wrong."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

import paged_kv_cache_store_gb300 as pa
from paged_kv_cache_store_gb300 import build as pabuild

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def L():
    pabuild.build()
    return pa.load_library()


def exact_turns(rotary, theta, scaling):
    """Turns per position times 2^64, to 50 digits."""
    getcontext().prec = 60
    theta, kind, out = Decimal(theta), scaling[0] if scaling else None, []
    s = Decimal(scaling[1]) if scaling else Decimal(1)
    if kind == "yarn":
        fast, slow = scaling[3:] if len(scaling) > 3 else (32.0, 1.0)
        dim = lambda beta: rotary * math.log(scaling[2] / (2 * math.pi * beta)) / (2 * math.log(float(theta)))
        lo, hi = max(0, math.floor(dim(fast))), min(rotary - 1, math.ceil(dim(slow)))
    base = theta * s ** (Decimal(rotary) / (rotary - 2)) if kind == "ntk" else theta
    for i in range(rotary // 2):
        f = base ** (Decimal(-2 * i) / rotary)
        if kind == "linear":
            f = f / s
        elif kind == "yarn":
            r = Decimal(min(max(i - lo, 0), max(hi - lo, 0))) / (hi - lo) if hi > lo else Decimal(int(i > lo))
            f = f * (1 - r) + f / s * r
        out.append(f / (2 * PI) * 2 ** 64)
    return out


@pytest.mark.parametrize("scaling", [None, ("linear", 3.7), ("ntk", 8.0), ("ntk", 1.0), ("yarn", 4.0, 32768.0),
                                     ("yarn", 16.0, 4096.0, 16.0, 2.0), ("yarn", 40.0, 4096.0), ("yarn", 3.0, 5.0),
                                     ("yarn", 3.0, 1e30)])
@pytest.mark.parametrize("theta", [1e4, 1e6, 5e5, 1.5, 1.0000001, 1e30, 1e300])
@pytest.mark.parametrize("rotary", [16, 48, 64, 128])
def test_rope_frequencies_to_the_last_bit(L, rotary, theta, scaling):
    """Half a unit of 2^-64 of a turn, and 2^-30 of one for arithmetic of 100 bits."""
    r = pa.rope_frequencies(rotary, theta, scaling, device="cpu")
    want = exact_turns(rotary, theta, scaling)
    got = [int(x) % (1 << 64) for x in r.freqs.tolist()]
    assert len(got) == len(want)
    assert max(abs(g - w) for g, w in zip(got, want)) <= Decimal("0.500000001")
