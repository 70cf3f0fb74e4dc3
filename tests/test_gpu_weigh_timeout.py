"""A wait of the tensor-core weighing that runs out (debug build: the first CTA
withholds the copies of one tile of keys, so nothing completes its barrier): the
sequences of that CTA's part are reported, the others' weights are as ever, and
the device stays usable."""

import time

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from test_gpu_weigh import Weigh

pytestmark = pytest.mark.gpu


def _withheld(a, j):
    dbg = sv.load_library(sv.DEBUG_LIB_PATH)
    before = a["weights"].clone()
    with sv.use_library(sv.DEBUG_LIB_PATH):
        sv.cache_weigh(**a)   # (its kernel is loaded by the first call)
    torch.cuda.synchronize()
    a["weights"].copy_(before)
    assert dbg.spec_debug_withhold_tile(j) == 0
    start = time.monotonic()
    try:
        with sv.use_library(sv.DEBUG_LIB_PATH):
            status = sv.cache_weigh(**a)["status"]
        torch.cuda.synchronize()
        # the wait that runs out, and the waits for the copies before the CTA ends
        assert time.monotonic() - start < 4.0
    finally:
        assert dbg.spec_debug_withhold_tile(-1) == 0
    return status


@pytest.mark.parametrize("D,N,j", [(128, 1, 0), (128, 9, 3), (64, 3, 1), (64, 2, 12)])
def test_the_first_part_is_reported(D, N, j):
    """The first CTA's part lies inside the first of 40 long sequences."""
    w = Weigh(91, [6000] * 40, N, 1, 2, D, 64, "bf16")
    a = w.args()
    assert _withheld(a, j).tolist() == [sv.SPEC_ETIMEOUT] + [0] * 39
    off = (a["weights"].double().cpu() - w.want).abs()
    assert (off <= w.tol)[1:].all()
    with sv.use_library(sv.DEBUG_LIB_PATH):
        w.check()
