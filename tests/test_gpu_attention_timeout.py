"""A wait of the tensor-core attention that runs out (debug build: the first CTA
withholds the copies of one tile, so nothing completes its barrier): the
sequences of that CTA's part are reported, the others are as ever, and the
device stays usable."""

import time

import numpy as np
import pytest
import torch

import paged
import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu


def _withheld(a, j):
    dbg = sv.load_library(sv.DEBUG_LIB_PATH)
    with sv.use_library(sv.DEBUG_LIB_PATH):
        sv.tree_attention(with_lse=True, **a)   # (its kernels are loaded by the first call)
    torch.cuda.synchronize()
    assert dbg.spec_debug_withhold_tile(j) == 0
    start = time.monotonic()
    try:
        with sv.use_library(sv.DEBUG_LIB_PATH):
            got = sv.tree_attention(with_lse=True, **a)
        torch.cuda.synchronize()
        # the wait that runs out, and the wait for that copy before the CTA ends
        assert time.monotonic() - start < 3.0
    finally:
        assert dbg.spec_debug_withhold_tile(-1) == 0
    return got


def _same(got, want, first):
    for k in ("out", "lse", "status"):
        assert torch.equal(got[k][first:], want[k][first:]), k


@pytest.mark.parametrize("D,j", [(128, 0), (128, 3), (64, 1), (64, 8)])
def test_one_long_part(D, j):
    """The first CTA's part lies inside the first of 40 long sequences."""
    a = paged.Case(81, [2000] * 40, 9, 2, 4, D, 64, "bf16", True).args()
    want = sv.tree_attention(with_lse=True, **a)
    got = _withheld(a, j)
    assert got["status"].tolist() == [3] + [0] * 39   # SPEC_ETIMEOUT
    _same(got, want, 1)
    with sv.use_library(sv.DEBUG_LIB_PATH):
        _same(sv.tree_attention(with_lse=True, **a), want, 0)


@pytest.mark.parametrize("D,G,j", [(128, 4, 0), (64, 16, 5)])
def test_a_part_of_many_sequences(D, G, j):
    lens = np.random.default_rng(82).integers(0, 100, 600)
    a = paged.Case(83, lens, 9, 2, G, D, 16, "bf16", True).args()
    want = sv.tree_attention(with_lse=True, **a)
    got = _withheld(a, j)
    st = got["status"].tolist()
    lost = st.index(0)
    assert 1 <= lost < 20 and st == [3] * lost + [0] * (600 - lost)
    _same(got, want, lost)
    with sv.use_library(sv.DEBUG_LIB_PATH):
        _same(sv.tree_attention(with_lse=True, **a), want, 0)


def test_release_builds_withhold_nothing():
    assert sv.load_library(sv.LIB_PATH).spec_debug_withhold_tile(0) == -1
