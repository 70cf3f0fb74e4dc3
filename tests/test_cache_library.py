"""The paged-cache entry points reject invalid arguments on the host (no GPU
needed: an invalid call returns SPEC_EINVAL before any CUDA call)."""

import ctypes
import os

import pytest

import speculative_decoding_verification_05_gb300 as sv

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below is invalid
ODD = ctypes.c_void_p((1 << 20) + 2)
EINVAL = 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sv.LIB_PATH):
        from speculative_decoding_verification_05_gb300 import build
        build.build()
    return sv.load_library()


def _cache(**k):
    a = dict(k=1 << 20, v=1 << 20, layers=1, num_pages=10, page_size=16, kv_heads=2, head_dim=64, layer_stride=0,
             page_stride=2048, token_stride=128, head_stride=64)
    a.update(k)
    return sv.SpecCache(*a.values())


BAD_CACHE = [dict(k=0), dict(v=0), dict(k=(1 << 20) + 8), dict(num_pages=0), dict(page_size=12), dict(page_size=4),
             dict(page_size=512), dict(kv_heads=0), dict(head_dim=0), dict(head_dim=12), dict(head_dim=264),
             dict(page_stride=2044), dict(token_stride=-128), dict(head_stride=65), dict(layers=0)]


def test_status_names(lib):
    assert lib.spec_status_string(6) == b"SPEC_ENOPAGES"


def _attention(lib, cache=None, **k):
    a = dict(q=FAKE, dtype=1, table=FAKE, stride=4, width=4, lens=FAKE, mask=None, n=None, B=2, N=3, Hq=4, scale=0.1,
             out=FAKE, lse=None, status=None, ws=FAKE, bytes=1 << 40)
    a.update(k)
    return lib.spec_tree_attention(a["q"], cache or _cache(), a["dtype"], a["table"], a["stride"], a["width"], a["lens"],
                                   a["mask"], a["n"], a["B"], a["N"], a["Hq"], a["scale"], a["out"], a["lse"],
                                   a["status"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=ctypes.c_void_p((1 << 20) + 8)), dict(dtype=5), dict(table=None), dict(stride=3),
    dict(width=0), dict(lens=None), dict(lens=ODD), dict(n=ODD), dict(B=0), dict(B=65536), dict(N=0), dict(N=1025),
    dict(Hq=3), dict(Hq=0), dict(Hq=258), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None),
    dict(out=ODD), dict(lse=ODD), dict(status=ODD), dict(ws=None), dict(ws=ctypes.c_void_p((1 << 20) + 16)),
    dict(bytes=1000)])
def test_attention_rejects_bad_arguments(lib, kw):
    assert _attention(lib, **kw) == EINVAL


@pytest.mark.parametrize("kw", BAD_CACHE + [dict(layers=2)])
def test_attention_rejects_bad_caches(lib, kw):
    assert _attention(lib, _cache(**kw)) == EINVAL


def test_attention_workspace(lib):
    w = lib.spec_tree_attention_workspace_size
    assert w(1, 5, 32, 8, 128, 1) > 0 and w(1, 5, 32, 8, 128, 1) % 256 == 0
    for bad in ((0, 5, 32, 8, 128, 1), (1, 0, 32, 8, 128, 1), (1, 5, 31, 8, 128, 1), (1, 5, 32, 8, 130, 1),
                (1, 5, 32, 8, 128, 3)):
        assert w(*bad) == 0


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=ODD), dict(table=None), dict(lens=None), dict(B=0), dict(N=0),
                                dict(N=(1 << 20) + 1), dict(n=ODD), dict(status=ODD)]
                         + [dict(cache=c) for c in BAD_CACHE + [dict(layers=2)]])
def test_append_rejects_bad_arguments(lib, kw):
    a = dict(k=FAKE, v=FAKE, cache={}, table=FAKE, lens=FAKE, n=None, B=2, N=3, status=None)
    a.update(kw)
    assert lib.spec_cache_append(a["k"], a["v"], _cache(**a["cache"]), 1, a["table"], 4, 4, a["lens"], a["n"], a["B"],
                                 a["N"], a["status"], None) == EINVAL


@pytest.mark.parametrize("kw", [dict(table=None), dict(lens=None), dict(acc=None), dict(path=ODD), dict(B=0), dict(W=0),
                                dict(W=1025), dict(new=None), dict(new=FAKE), dict(new=ctypes.c_void_p((1 << 20) - 4)),
                                dict(status=ODD)] + [dict(cache=c) for c in BAD_CACHE])
def test_compact_rejects_bad_arguments(lib, kw):
    a = dict(cache={}, table=FAKE, lens=FAKE, acc=FAKE, path=FAKE, B=2, W=3, new=ctypes.c_void_p(1 << 21), status=None)
    a.update(kw)
    assert lib.spec_cache_compact(_cache(**a["cache"]), 1, a["table"], 4, 4, a["lens"], a["acc"], a["path"], a["B"],
                                  a["W"], a["new"], a["status"], None) == EINVAL


@pytest.mark.parametrize("kw", [dict(table=None), dict(stride=2), dict(width=0), dict(S=0), dict(refs=None),
                                dict(refs=ODD), dict(P=0), dict(ps=10), dict(seqs=ODD), dict(tok=None), dict(F=0),
                                dict(F=9), dict(S=5000, F=4097), dict(status=ODD)])
def test_resize_rejects_bad_arguments(lib, kw):
    a = dict(table=FAKE, stride=4, width=4, S=8, refs=FAKE, P=10, ps=16, seqs=None, tok=FAKE, F=3, status=None)
    a.update(kw)
    assert lib.spec_cache_resize(a["table"], a["stride"], a["width"], a["S"], a["refs"], a["P"], a["ps"], a["seqs"],
                                 a["tok"], a["F"], a["status"], None) == EINVAL


@pytest.mark.parametrize("kw", [dict(table=None), dict(S=0), dict(refs=None), dict(lens=None), dict(src=None),
                                dict(dst=ODD), dict(F=0), dict(F=9), dict(ws=None), dict(bytes=8)]
                         + [dict(cache=c) for c in BAD_CACHE])
def test_fork_rejects_bad_arguments(lib, kw):
    a = dict(cache={}, table=FAKE, S=8, refs=FAKE, lens=FAKE, src=FAKE, dst=FAKE, F=3, ws=FAKE, bytes=1 << 20)
    a.update(kw)
    assert lib.spec_cache_fork(_cache(**a["cache"]), 1, a["table"], 4, 4, a["S"], a["refs"], a["lens"], a["src"],
                               a["dst"], a["F"], None, a["ws"], a["bytes"], None) == EINVAL
    assert lib.spec_cache_fork_workspace_size(0) == 0 and lib.spec_cache_fork_workspace_size(3) >= 48
