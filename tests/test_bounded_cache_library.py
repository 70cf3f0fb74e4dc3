"""The rotary append, the weighing and the eviction reject invalid arguments on
the host (no GPU needed: an invalid call returns SPEC_EINVAL before any CUDA call)."""

import ctypes
import os

import pytest

import speculative_decoding_verification_05_gb300 as sv
from test_cache_library import BAD_CACHE, _cache

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below is invalid
FAR = ctypes.c_void_p(1 << 40)
ODD = ctypes.c_void_p((1 << 20) + 2)
EINVAL = 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sv.LIB_PATH):
        from speculative_decoding_verification_05_gb300 import build
        build.build()
    return sv.load_library()


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=ctypes.c_void_p((1 << 20) + 8)), dict(k=None), dict(v=ODD), dict(dtype=5), dict(table=None), dict(stride=3),
    dict(lens=None), dict(turns=None), dict(turns=ctypes.c_void_p((1 << 20) + 4)), dict(dim=0), dict(dim=3), dict(dim=66),
    dict(factor=float("nan")), dict(factor=float("inf")), dict(pos=ODD), dict(depth=ODD), dict(n=ODD), dict(B=0), dict(B=65536),
    dict(N=0), dict(N=(1 << 20) + 1), dict(Hq=0), dict(out=None), dict(out=FAKE), dict(out=ctypes.c_void_p((1 << 20) + 64)),
    dict(out=ctypes.c_void_p((1 << 20) - 64)), dict(status=ODD)] + [dict(cache=c) for c in BAD_CACHE + [dict(layers=2)]])
def test_append_rotary(lib, kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, cache={}, dtype=1, table=FAKE, stride=4, width=4, lens=FAKE, turns=FAKE, dim=64, factor=1.0,
             pos=None, depth=None, n=None, B=2, N=3, Hq=4, out=FAR, status=None)
    a.update(kw)
    assert lib.spec_cache_append_rotary(a["q"], a["k"], a["v"], _cache(**a["cache"]), a["dtype"], a["table"], a["stride"], a["width"],
                                        a["lens"], a["turns"], a["dim"], 0, a["factor"], a["pos"], a["depth"], a["n"], a["B"],
                                        a["N"], a["Hq"], a["out"], a["status"], None) == EINVAL


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=ODD), dict(lse=None), dict(lse=ODD), dict(dtype=5), dict(table=None), dict(width=0), dict(lens=None),
    dict(acc=ODD), dict(path=ODD), dict(path=FAKE, acc=None), dict(path=FAKE, W=0), dict(path=FAKE, W=1025), dict(B=0), dict(N=0),
    dict(N=1025), dict(Hq=3), dict(Hq=258), dict(scale=float("nan")), dict(w=None), dict(w=ODD), dict(cap=0), dict(cap=(1 << 31) + 1),
    dict(status=ODD)] + [dict(cache=c) for c in BAD_CACHE + [dict(layers=2)]])
def test_weigh(lib, kw):
    a = dict(q=FAKE, lse=FAKE, cache={}, dtype=1, table=FAKE, width=4, lens=FAKE, acc=FAKE, path=None, B=2, N=3, W=3, Hq=4, scale=0.1,
             w=FAKE, cap=100, status=None)
    a.update(kw)
    assert lib.spec_cache_weigh(a["q"], a["lse"], _cache(**a["cache"]), a["dtype"], a["table"], 4, a["width"], a["lens"], a["acc"],
                                a["path"], a["B"], a["N"], a["W"], a["Hq"], a["scale"], a["w"], a["cap"], a["status"], None) == EINVAL


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(lens=None), dict(budget=None), dict(budget=ODD), dict(sink=-1), dict(recent=-1), dict(w=None), dict(w=ODD),
    dict(cap=0), dict(B=0), dict(new=None), dict(new=FAKE), dict(status=ctypes.c_void_p((1 << 20) + 4)), dict(new=ctypes.c_void_p(1 << 41)),
    dict(status=FAR), dict(status=ODD), dict(ws=None), dict(ws=ctypes.c_void_p((1 << 20) + 16)), dict(bytes=1000)]
    + [dict(cache=c) for c in BAD_CACHE])
def test_evict(lib, kw):
    a = dict(cache={}, table=FAKE, lens=FAKE, budget=ctypes.c_void_p(1 << 41), sink=1, recent=1, w=FAKE, cap=100, B=2, new=FAR,
             status=None, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    assert lib.spec_cache_evict(_cache(**a["cache"]), 1, a["table"], 4, 4, a["lens"], a["budget"], a["sink"], a["recent"], a["w"],
                                a["cap"], a["B"], a["new"], a["status"], a["ws"], a["bytes"], None) == EINVAL


def test_evict_workspace(lib):
    w = lib.spec_cache_evict_workspace_size
    assert w(2, 3, 4, 100) >= 2 * 3 * 4 * 408 and w(2, 3, 4, 100) % 256 == 0
    for bad in ((0, 3, 4, 100), (2, 0, 4, 100), (2, 70000, 4, 100), (2, 3, 0, 100), (2, 3, 4, 0), (1 << 20, 1 << 12, 4, 100)):
        assert w(*bad) == 0
