"""Rotary frequencies: host arithmetic of the library, against the formulas in
extended precision, and the binding's handle."""

import ctypes
import math
import os
from decimal import Decimal, getcontext

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv

getcontext().prec = 60
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sv.LIB_PATH):
        from speculative_decoding_verification_05_gb300 import build
        build.build()
    return sv.load_library()


def frequencies(dim, base, scaling, s, original):
    """Radians a position and the factor, by the formulas."""
    base, s = Decimal(base), Decimal(s)
    if scaling == "ntk":
        base = base * (s.ln() * Decimal(dim) / Decimal(dim - 2)).exp()
    f = [(base.ln() * Decimal(-2 * j) / Decimal(dim)).exp() for j in range(dim // 2)]
    factor = 1.0
    if scaling == "linear":
        f = [x / s for x in f]
    if scaling == "yarn":
        pair = lambda r: dim * math.log(original / (r * 2 * math.pi)) / (2 * math.log(float(base)))
        lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), dim - 1)
        keep = [1 - (j - lo) / max(hi - lo, 0.001) for j in range(dim // 2)]
        factor = 0.1 * math.log(float(s)) + 1.0
    if scaling == "bands":
        keep = [(original / (2 * math.pi / float(x)) - 1) / 3 for x in f]
    if scaling in ("yarn", "bands"):
        keep = [Decimal(min(max(k, 0.0), 1.0)) for k in keep]
        f = [x * k + x / s * (1 - k) for x, k in zip(f, keep)]
    return f, factor


@pytest.mark.parametrize("dim,base", [(2, 10000.0), (24, 10000.0), (64, 500000.0), (128, 10000.0), (256, 1e6)])
@pytest.mark.parametrize("scaling,s,original", [(None, 1, 0), ("linear", 4, 0), ("ntk", 8, 0), ("yarn", 16, 4096),
                                                ("bands", 8, 8192), ("yarn", 1, 64), ("bands", 1.5, 3)])
def test_turns(lib, dim, base, scaling, s, original):
    if scaling == "ntk" and dim == 2:
        return
    r = sv.rotary(dim, base, scaling=scaling, scale=s, original=original, device="cpu")
    f, factor = frequencies(dim, base, scaling, s, original)
    assert r.turns.shape == (dim // 2,) and r.turns.dtype is torch.int64 and not r.interleaved
    assert abs(r.factor - factor) <= 2.0 ** -23
    for got, x in zip(r.turns.tolist(), f):
        want = x / TWO_PI * 2 ** 64
        # pow, the mix and the division: a few roundings of 2^-53, and pow's exponent (at most ln base ln 2^.. < 2^6 of them)
        assert abs((got % 2 ** 64) - want) <= want * Decimal(2.0 ** -45) + 1


def test_given_frequencies(lib):
    f = [1.0, 0.5, 2 * math.pi, 7.0, -1.0]
    r = sv.rotary(10, frequencies=f, interleaved=True, device="cpu")
    assert r.interleaved and r.factor == 1.0
    for got, x in zip(r.turns.tolist(), f):
        assert abs((got / 2.0 ** 64 - x / (2 * math.pi) + 0.5) % 1.0 - 0.5) < 1e-14
    assert torch.equal(sv.rotary(10, frequencies=torch.tensor(f, dtype=torch.float64), device="cpu").turns, r.turns)
    for bad in (dict(frequencies=[1.0]), dict(frequencies=[math.nan] * 5), dict(frequencies=[math.inf] * 5),
                dict(frequencies=1.0), dict(frequencies=f, scaling="linear")):
        with pytest.raises(sv.SpecError):
            sv.rotary(10, device="cpu", **bad)


@pytest.mark.parametrize("kw", [
    dict(dim=0), dict(dim=3), dict(dim=258), dict(base=1.0), dict(base=0.0), dict(base=math.nan), dict(base=math.inf),
    dict(scaling="linear", scale=0.5), dict(scaling="linear", scale=math.inf), dict(scaling="ntk", scale=math.nan),
    dict(scaling="ntk", dim=2, scale=2.0), dict(scaling="yarn", scale=2.0), dict(scaling="bands", scale=2.0, original=-1.0),
    dict(scaling="yarn", scale=2.0, original=math.inf), dict(scaling="ntk", scale=1e300), dict(scaling="other")])
def test_refusals(lib, kw):
    with pytest.raises(sv.SpecError):
        sv.rotary(**{"dim": 64, "device": "cpu", **kw})
    assert lib.spec_rotary_turns(64, 10000.0, 7, 1.0, 0.0, (ctypes.c_uint64 * 32)(), ctypes.c_float()) == sv.SPEC_EINVAL
