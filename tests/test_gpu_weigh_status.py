"""The statuses of the weighing: whatever the array held, good sequences are 0, bad ones
SPEC_EDATA, and what a part that gave up reports stays, also where other work on the GPU makes
the checking blocks of its sequences late."""

import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from test_gpu_weigh import Weigh

pytestmark = pytest.mark.gpu


def _call(a, status, path=None):
    """spec_cache_weigh of the arguments of ``cache_weigh`` into a given status array."""
    lib = sv.load_library(path)
    B, N, Hq, D = a["q"].shape
    cache, _, dt = sv._cache_args(a["k_cache"], a["k_cache"], 0)
    rc = lib.spec_cache_weigh(a["q"].data_ptr(), a["lse"].data_ptr(), cache, dt, a["page_table"].data_ptr(),
                              a["page_table"].shape[1], a["page_table"].shape[1], a["cache_len"].data_ptr(), None, None, B, N,
                              N, Hq, a["scale"], a["weights"].data_ptr(), a["weights"].shape[-1],
                              None if status is None else status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (96, "bf16"), (64, "f32")])
def test_whatever_the_array_held(D, dtype):
    w = Weigh(31, [70] * 200, 2, 1, 2, D, 16, dtype)
    a = w.args()
    a["page_table"][5, 3] = -1
    a["page_table"][199, 0] = 10 ** 6
    a["cache_len"][77] = -3
    want = [sv.SPEC_EDATA if b in (5, 77, 199) else 0 for b in range(200)]
    for held in (0, 77, -1, -2 ** 31, 2 ** 31 - 1):
        status = torch.full((200,), held, dtype=torch.int32, device="cuda")
        _call(a, status)
        assert status.tolist() == want
    _call(a, None)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(a, status)
    for held in (77, -1):
        status.fill_(held)
        g.replay()
        torch.cuda.synchronize()
        assert status.tolist() == want


def test_a_timeout_stays():
    """Two calls on two streams whose first parts give up, each over 200 sequences that other blocks
    check; some of either call's blocks start only when the other's first one has ended."""
    dbg = sv.load_library(sv.DEBUG_LIB_PATH)
    w = [Weigh(32 + i, [70] * 400, 1, 2, 2, 128, 16, "bf16") for i in range(2)]
    args = [x.args() for x in w]
    streams = [torch.cuda.Stream() for _ in w]
    status = [torch.full((400,), -1, dtype=torch.int32, device="cuda") for _ in w]
    _call(args[0], status[0], sv.DEBUG_LIB_PATH)   # (the kernel is loaded by the first call)
    args[0]["weights"].copy_(w[0].w)
    torch.cuda.synchronize()
    assert dbg.spec_debug_withhold_tile(0) == 0
    try:
        for a, s, st in zip(args, streams, status):
            with torch.cuda.stream(s):
                _call(a, st, sv.DEBUG_LIB_PATH)
        torch.cuda.synchronize()
    finally:
        assert dbg.spec_debug_withhold_tile(-1) == 0
    for x, a, st in zip(w, args, status):
        st = st.tolist()
        lost = st.index(0)
        assert 1 <= lost < 20 and st == [sv.SPEC_ETIMEOUT] * lost + [0] * (400 - lost)
        off = (a["weights"].double().cpu() - x.want).abs()
        assert (off <= x.tol)[lost:].all()
