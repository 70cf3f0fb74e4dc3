"""token_logprobs rejects invalid arguments on the host (no GPU needed: an
invalid call returns SPEC_EINVAL before any CUDA call)."""

import ctypes
import os

import pytest

import speculative_decoding_verification_05_gb300 as sv

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below is invalid
ODD = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sv.LIB_PATH):
        from speculative_decoding_verification_05_gb300 import build
        build.build()
    return sv.load_library()


@pytest.mark.parametrize("kw", [
    dict(z=None), dict(z=ODD), dict(dtype=2), dict(tok=None), dict(tok=ODD), dict(B=0), dict(B=(1 << 24) + 1), dict(P=0),
    dict(P=65537), dict(B=1 << 12, P=(1 << 16)), dict(V=0), dict(V=(1 << 18) + 1), dict(T=0.0), dict(T=-1.0),
    dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-42), dict(T=3e38, top=33), dict(top=-1), dict(top=33),
    dict(V=4, top=5), dict(lp=None), dict(lp=ODD), dict(rank=ODD), dict(ent=ODD), dict(tt=None), dict(tl=None),
    dict(tt=ODD), dict(tl=ODD), dict(status=ODD)])
def test_rejects_bad_arguments(lib, kw):
    a = dict(z=FAKE, dtype=0, tok=FAKE, B=2, P=3, V=100, T=1.0, top=4, lp=FAKE, rank=None, ent=None, tt=FAKE, tl=FAKE,
             status=None)
    a.update(kw)
    assert lib.spec_token_logprobs(a["z"], a["dtype"], a["tok"], a["B"], a["P"], a["V"], a["T"], a["top"], a["lp"],
                                   a["rank"], a["ent"], a["tt"], a["tl"], a["status"], None) == sv.SPEC_EINVAL
