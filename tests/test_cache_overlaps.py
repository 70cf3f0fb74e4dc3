"""spec_cache_compact refuses outputs that overlap its inputs (no GPU needed: the
call returns SPEC_EINVAL before any CUDA call)."""

import ctypes

import pytest

from test_cache_library import EINVAL, _cache, lib  # noqa: F401

AT = dict(lens=1 << 20, acc=2 << 20, path=3 << 20, new=4 << 20, status=5 << 20)   # never dereferenced


@pytest.mark.parametrize("out,other,ints", [(o, i, n) for o in ("new", "status") for i, n in (
    ("lens", 5), ("acc", 5), ("path", 15), ("new", 5), ("status", 5)) if o != i])
def test_compact_refuses_overlapping_outputs(lib, out, other, ints):  # noqa: F811
    def call(**k):
        a = {n: ctypes.c_void_p(x) for n, x in {**AT, **k}.items()}
        return lib.spec_cache_compact(_cache(), 1, ctypes.c_void_p(6 << 20), 4, 4, a["lens"], a["acc"], a["path"], 5, 3,
                                      a["new"], a["status"], None)

    for at in (0, 4 * (ints - 1), -16):
        assert call(**{out: AT[other] + at}) == EINVAL
