"""Tree attention where a core goes through many sequences, heads and row tiles
in one launch: ragged lengths that end in either half of a tile, whole and
shared units, masks at odd addresses. Against the definition in 64 bits;
tolerances: paged.Case.expected."""

import numpy as np
import pytest
import torch

import paged
import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu


def _lens(seed, B, hi):
    """Lengths of every size up to hi, the tile's own edges among them."""
    x = np.random.default_rng(seed).integers(0, hi + 1, B)
    edges = [e for e in (0, 1, 62, 63, 64, 65, 126, 127, 128, 129, 191, 192, 256) if e <= hi]
    x[:len(edges)] = edges[:B]
    return np.random.default_rng(seed + 1).permutation(x)


# B, longest, N, kv heads, group, D, page size, tree
BATCHES = [
    (90, 700, 1, 8, 4, 128, 64, False),
    (90, 700, 1, 8, 4, 64, 16, False),
    (40, 300, 6, 12, 1, 64, 16, True),
    (16, 500, 64, 8, 1, 128, 16, True),
    (20, 400, 40, 2, 8, 128, 32, True),
    (20, 400, 40, 2, 8, 64, 8, True),
    (24, 300, 33, 3, 7, 128, 16, True),
    (8, 200, 150, 2, 2, 64, 128, True),
    (60, 400, 3, 6, 3, 96, 16, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_many_units_a_core(i, dtype):
    B, hi, N, H, G, D, ps, tree = BATCHES[i]
    counts = np.where(np.arange(B) % 4 == 3, (2 * N) // 3, N)
    c = paged.Case(300 + i, _lens(i, B, hi), N, H, G, D, ps, dtype, tree, counts)
    got = sv.tree_attention(with_lse=True, **c.args())
    assert got["status"].tolist() == [0] * B
    paged.assert_attention(got, c.expected(), f"batch {i}")


@pytest.mark.parametrize("N,G", [(20, 1), (9, 7), (64, 1), (65, 1), (33, 4)])
@pytest.mark.parametrize("D", [8, 64, 72, 136, 192, 256])
def test_many_rows_on_the_cuda_cores(D, N, G):
    """Row tiles that are partly filled, head sizes of every column grouping, few and many keys, both types."""
    for dtype in ("f32", "bf16"):
        c = paged.Case(800 + N, [0, 1, 63, 64, 200, 700], N, 2, G, D, 16, dtype, True, counts=[N, 1, N - 1, N, 0, N])
        got = sv.tree_attention(with_lse=True, **c.args())
        assert got["status"].tolist() == [0] * 6
        paged.assert_attention(got, c.expected(), f"D {D} N {N} G {G} {dtype}")


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scales_that_are_not_positive(scale):
    for D, dtype in ((64, "bf16"), (128, "bf16"), (128, "f32")):
        c = paged.Case(850, [90, 0, 300], 30, 2, 3, D, 16, dtype, True, counts=[30, 9, 1])
        c.scale = scale
        got = sv.tree_attention(with_lse=True, **c.args())
        paged.assert_attention(got, c.expected(), f"D {D} {dtype} {scale}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,G,hi,ps", [(1, 1, 1, 1, 60, 16), (12, 3, 8, 1, 400, 16), (19, 5, 8, 2, 100, 32),
                                            (20, 5, 8, 2, 100, 32), (2, 60, 8, 8, 430, 64), (38, 2, 4, 4, 120, 128),
                                            (30, 1, 5, 4, 511, 256)])
def test_few_short_units(B, N, H, G, hi, ps, dtype):
    """Units of a few tiles, up to as many as there are cores: split and whole ones, and the same sequences in a
    table whose width allows for long ones."""
    for D in (64, 128):
        c = paged.Case(700 + B, _lens(B, B, hi), N, H, G, D, ps, dtype, True)
        want = c.expected()
        a = c.args()
        got = sv.tree_attention(with_lse=True, **a)
        assert got["status"].tolist() == [0] * B
        paged.assert_attention(got, want, f"B {B} D {D}")
        wide = torch.full((B, 3000), -1, dtype=torch.int32, device="cuda")
        wide[:, :c.M] = a["page_table"]
        a["page_table"] = wide
        got = sv.tree_attention(with_lse=True, **a)
        assert got["status"].tolist() == [0] * B
        paged.assert_attention(got, want, f"B {B} D {D}, wide table")


@pytest.mark.parametrize("rows", range(1, 18))
def test_every_row_count_of_a_core_tile(rows):
    """float32: the warps' shares of rows and positions; head sizes of one and two column blocks a lane."""
    for D in (8, 64, 72, 128, 136, 256):
        c = paged.Case(400 + rows, [rows, 150], rows, 2, 1, D, 16, "f32", True)
        got = sv.tree_attention(with_lse=True, **c.args())
        assert got["status"].tolist() == [0, 0]
        paged.assert_attention(got, c.expected(), f"rows {rows} D {D}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_masks_at_any_address(shift, dtype):
    c = paged.Case(500 + shift, [100, 61, 0], 61, 2, 2, 128, 16, dtype, True, counts=[61, 40, 7])
    a = c.args()
    store = torch.full((a["mask"].numel() + shift,), 255, dtype=torch.uint8, device="cuda")
    a["mask"] = store[shift:].view(a["mask"].shape).copy_(a["mask"])
    got = sv.tree_attention(with_lse=True, **a)
    paged.assert_attention(got, c.expected(), f"mask at {shift}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_index_checks_of_the_debug_build(dtype):
    """The same bits from the build with device-side index checks, and none of them fails."""
    import ctypes

    dbg = sv.load_library(sv.DEBUG_LIB_PATH)

    def step():
        g = np.random.default_rng(601)
        c = paged.Case(602, _lens(603, 24, 300), 9, 2, 4, 64 if g.integers(2) else 128, 16, dtype, True)
        a = c.args()
        out = sv.tree_attention(with_lse=True, **a)
        k, v = (x[None].clone() for x in (a["k_cache"], a["v_cache"]))
        new = torch.from_numpy(g.standard_normal((24, 9, 2, c.D), dtype=np.float32)).to(paged.TD[dtype]).cuda()
        app = sv.cache_append(new, -new, k[0], v[0], a["page_table"], a["cache_len"], a["n_nodes"])
        acc = torch.from_numpy(g.integers(0, 3, 24).astype(np.int32)).cuda()
        path = torch.tensor([[0, 3, 7]], dtype=torch.int32, device="cuda").repeat(24, 1)
        path.masked_fill_(torch.arange(3, device="cuda") > acc[:, None], -1)
        com = sv.cache_compact(k, v, a["page_table"], a["cache_len"], acc, path)
        table, refs = torch.full((6, 8), -1, dtype=torch.int32, device="cuda"), torch.zeros(c.P, dtype=torch.int32, device="cuda")
        lens = torch.zeros(6, dtype=torch.int32, device="cuda")
        seqs = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
        res = sv.cache_resize(table, refs, seqs(0, 1), seqs(40, 100), 16)
        lens[:2] = seqs(40, 100)
        frk = sv.cache_fork(k, v, table, lens, refs, seqs(0, 0, 1), seqs(2, 3, 4))
        end = sv.cache_resize(table, refs, seqs(0, 3), seqs(0, 17), 16)
        torch.cuda.synchronize()
        return [out["out"], out["lse"], k, v, com["cache_len"], table, refs, lens] + \
            [x["status"] for x in (out, app, com, res, frk, end)]

    release = step()
    with sv.use_library(sv.DEBUG_LIB_PATH):
        checked = step()
    assert dbg.spec_debug_failures(ctypes.byref(ctypes.c_int(0))) == 0
    for a, b in zip(release, checked):
        assert torch.equal(a, b)
