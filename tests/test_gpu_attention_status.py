"""The statuses of the tensor-core attention: whatever the array held, good sequences are 0, bad
ones SPEC_EDATA, and what a part that gave up reports stays, whichever of the grid's blocks runs
when. Whole units (few, short: one kernel) and shared ones (a second kernel joins them)."""

import numpy as np
import pytest
import torch

import paged
import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu
# sequences, longest context, key heads: units of their parts alone, and shared ones
SHAPES = {"whole": (100, 300, 1), "shared": (120, 900, 2)}


def _case(kind, seed, D=128):
    B, most, H = SHAPES[kind]
    lens = np.random.default_rng(seed).integers(100, most, B)
    return paged.Case(seed, lens, 3, H, 2, D, 16, "bf16", False)


@pytest.mark.parametrize("kind", SHAPES)
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (64, "f32")])
def test_whatever_the_array_held(kind, D, dtype):
    c = _case(kind, 1, D)
    c.dtype, c.k, c.v, c.q = dtype, c.k.to(paged.TD[dtype]), c.v.to(paged.TD[dtype]), c.q.to(paged.TD[dtype])
    a = c.args()
    a["page_table"][5, 3] = -1
    a["page_table"][99, 0] = 10 ** 6
    a["cache_len"][77] = -3
    a["n_nodes"][8] = 0
    want = [sv.SPEC_EDATA if b in (5, 77, 99) else 0 for b in range(c.B)]
    o = {"status": torch.empty(c.B, dtype=torch.int32, device="cuda")}
    first = None
    for held in (0, 77, -1, -2 ** 31, 2 ** 31 - 1):
        o["status"].fill_(held)
        r = sv.tree_attention(out=o, with_lse=True, **a)
        assert r["status"].data_ptr() == o["status"].data_ptr() and r["status"].tolist() == want
        first = first or r
        for k in ("out", "lse"):
            assert torch.equal(r[k].nan_to_num(9.0), first[k].nan_to_num(9.0))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.tree_attention(out=o, **a)
    for held in (77, -1):
        o["status"].fill_(held)
        g.replay()
        torch.cuda.synchronize()
        assert o["status"].tolist() == want


@pytest.mark.parametrize("kind", SHAPES)
@pytest.mark.parametrize("j", [0, 3])
def test_a_timeout_stays(kind, j):
    """Two calls on two streams whose first parts give up; some of either call's blocks start only
    when the other's first one has ended."""
    dbg = sv.load_library(sv.DEBUG_LIB_PATH)
    args = [_case(kind, 2 + i).args() for i in range(2)]
    B = SHAPES[kind][0]
    want = [sv.tree_attention(with_lse=True, **a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    with sv.use_library(sv.DEBUG_LIB_PATH):
        for a in args:
            sv.tree_attention(with_lse=True, **a)   # (the kernels are loaded by the first call)
        torch.cuda.synchronize()
        assert dbg.spec_debug_withhold_tile(j) == 0
        try:
            got = []
            for a, s in zip(args, streams):
                with torch.cuda.stream(s):
                    o = {"status": torch.full((B,), -1, dtype=torch.int32, device="cuda")}
                    got.append(sv.tree_attention(with_lse=True, out=o, **a))
            torch.cuda.synchronize()
        finally:
            assert dbg.spec_debug_withhold_tile(-1) == 0
    for r, w in zip(got, want):
        st = r["status"].tolist()
        lost = st.index(0)
        assert 1 <= lost < 20 and st == [sv.SPEC_ETIMEOUT] * lost + [0] * (B - lost)
        for k in ("out", "lse"):
            assert torch.equal(r[k][lost:], w[k][lost:]), k
