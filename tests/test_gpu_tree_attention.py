"""Tree attention over a paged cache (spec_tree_attention) against its
definition in 64 bits: head layouts, page sizes, ragged lengths, masks that
leave a row empty, unseen NaN and infinities, memory orders, bad data, streams,
graphs and repeatability. Tolerances: paged.Case.expected."""

import math

import numpy as np
import pytest
import torch

import paged
import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu


def _run(c, **over):
    a = c.args()
    a.update(over)
    return sv.tree_attention(with_lse=True, **a)


def _check(c, label="", **over):
    got = _run(c, **over)
    assert got["status"].tolist() == [0] * c.B, label
    paged.assert_attention(got, c.expected(), label)
    return got


# lens, N, kv heads, group, D, page size, counts
SHAPES = [
    ([0], 1, 1, 1, 64, 16, None),
    ([1], 1, 1, 1, 128, 16, None),
    ([0, 1, 15, 16, 17], 1, 2, 4, 128, 16, None),
    ([127, 128, 129, 255, 256, 257], 1, 2, 8, 128, 64, None),
    ([63, 64, 65, 500], 5, 2, 4, 64, 8, None),
    ([1000], 5, 8, 4, 128, 16, None),
    ([0, 300, 7], 64, 2, 4, 128, 16, [64, 1, 33]),
    ([90, 0, 200], 33, 3, 7, 128, 32, [33, 0, 20]),
    ([40, 130], 130, 1, 3, 64, 128, [130, 129]),
    ([700, 5], 17, 1, 16, 128, 64, None),
    ([33], 3, 1, 128, 64, 16, None),
    ([100, 20], 9, 2, 2, 8, 16, None),
    ([100, 20], 9, 2, 2, 40, 16, None),
    ([257, 20], 9, 2, 5, 96, 256, None),
    ([150, 20], 20, 2, 5, 256, 16, None),
    ([2500, 4000], 2, 2, 2, 128, 16, None),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_matches_the_definition(i, tree, dtype):
    lens, N, H, G, D, ps, counts = SHAPES[i]
    _check(paged.Case(100 + i, lens, N, H, G, D, ps, dtype, tree, counts), f"shape {i}")


@pytest.mark.parametrize("D", [64, 128])
def test_large_tree_and_long_context(D):
    """A tree of 600 nodes: several row tiles, and tail tiles that hold nodes only."""
    _check(paged.Case(5, [77], 600, 1, 2, D, 32, "bf16", True))
    _check(paged.Case(6, [20011], 7, 1, 3, D, 64, "bf16", True))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_peaked_scores(dtype):
    """Scores tens of octaves apart: the running maximum moves by much more than any slack."""
    _check(paged.Case(7, [600, 900], 20, 2, 4, 128, 16, dtype, True, q_scale=12.0))
    # the largest keys last, so that each tile raises the maximum
    c = paged.Case(8, [640], 8, 1, 4, 64, 16, dtype, False)
    for t in range(640):
        c.k[c.table[0, t // 16], t % 16] *= 0.2 + 4.0 * t / 640
    _check(c)


@pytest.mark.parametrize("layout", ["hnd", "wide"])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_memory_orders(layout, D):
    _check(paged.Case(9, [70, 300], 13, 3, 4, D, 16, "bf16", True, layout=layout))
    _check(paged.Case(9, [70, 300], 13, 3, 2, D, 32, "f32", False, layout=layout))


def test_table_view_and_missing_counts():
    """A page table that is a view of a wider one; counts left out."""
    c = paged.Case(10, [70, 300, 5], 6, 2, 4, 128, 16, "bf16", True)
    wide = torch.full((3, c.M + 9), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.M] = torch.from_numpy(c.table)
    _check(c, page_table=wide[:, 2:2 + c.M], n_nodes=None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), -3e38])
def test_unseen_positions_do_not_reach_the_outputs(dtype, garbage):
    """Whatever lies past a sequence's end, in other pages, and in the nodes
    that a row's mask leaves out."""
    c = paged.Case(11, [50, 0, 130], 40, 2, 4, 128, 16, dtype, True, counts=[40, 9, 25], garbage=garbage)
    _check(c, "past the end")
    # node 7 of sequence 0 is itself unusable: only its descendants (and itself) may notice
    want = c.expected()
    t = int(c.lens[0]) + 7
    p, s = c.table[0, t // 16], t % 16
    c.k[p, s] = garbage
    c.v[p, s] = garbage
    got = _run(c)
    seen = torch.from_numpy(c.mask[0, :, 7] != 0)
    for k in ("out", "lse"):
        assert torch.isfinite(got[k][0][~seen].float()).all(), k
    clean = tuple(x.clone() for x in want)
    for x in (clean[0], clean[1]):
        x[0][seen] = 0
    got = {k: got[k].clone() for k in ("out", "lse")}
    for x in got.values():
        x[0][seen.cuda()] = 0
    paged.assert_attention(got, clean, "siblings of an unusable node")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_seen_values_that_are_not_finite_show(dtype):
    """An infinity or NaN in one element of a node's values: in exactly that
    output column of the rows that see the node."""
    c = paged.Case(12, [60, 3], 20, 1, 4, 128, 16, dtype, True)
    want = c.expected()
    for node, col, x in ((5, 3, float("inf")), (9, 100, float("-inf")), (2, 64, float("nan"))):
        t = int(c.lens[0]) + node
        c.v[c.table[0, t // 16], t % 16, 0, col] = x
    out = _run(c)["out"].double().cpu()
    for node, col, x in ((5, 3, float("inf")), (9, 100, float("-inf")), (2, 64, float("nan"))):
        seen = torch.from_numpy(c.mask[0, :, node] != 0)
        hit = out[0, seen][..., col]
        assert (torch.isnan(hit) if math.isnan(x) else hit == x).all()
        want[0][0, seen, :, col] = 0
        out[0, seen, :, col] = 0
    assert ((out - want[0]).abs() <= want[2]).all()


def test_a_row_that_sees_nothing():
    c = paged.Case(13, [0, 40], 12, 2, 4, 128, 16, "bf16", True)
    c.mask[0, 5] = 0
    c.mask[1, 7] = 0
    got = _check(c)
    assert (got["out"][0, 5] == 0).all() and torch.isneginf(got["lse"][0, 5]).all()
    assert (got["out"][1, 7] != 0).any()
    c.mask[0] = 0
    got = _check(c)
    assert (got["out"][0] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_data_is_reported_per_sequence(dtype):
    c = paged.Case(14, [100, 300, 40, 200, 10, 60], 8, 2, 4, 128, 16, dtype, True)
    a = c.args()
    a["page_table"][1, 3] = c.P          # no such page
    a["page_table"][3, 0] = -1
    a["cache_len"][2] = -1
    a["n_nodes"][4] = 9                  # above N
    a["cache_len"][5] = 16 * c.M         # past the table
    got = sv.tree_attention(with_lse=True, **a)
    assert got["status"].tolist() == [0, 4, 4, 4, 4, 4]
    assert torch.isnan(got["out"][1:].float()).all() and torch.isnan(got["lse"][1:]).all()
    want = tuple(x[:1] for x in c.expected())
    paged.assert_attention({k: got[k][:1] for k in ("out", "lse")}, want)


def test_offsets_past_32_bits():
    """Pages more than 2^32 bytes (and 2^31 elements) into the cache."""
    c = paged.Case(15, [200], 9, 8, 2, 128, 64, "bf16", True, spare=0)
    per_page = 64 * 8 * 128
    far = (1 << 32) // per_page + 11      # page far: element offset above 2^32
    k, v = (torch.empty(far + c.P, 64, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[far:], v[far:] = c.k.cuda(), c.v.cuda()
    _check(c, k_cache=k, v_cache=v, page_table=torch.from_numpy(c.table + far).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_and_streams_agree(dtype):
    """The same bits from repeated calls, from another stream and from a captured graph."""
    c = paged.Case(16, [3000, 700, 20], 20, 4, 4, 128, 16, dtype, True)
    a = c.args()
    first = sv.tree_attention(with_lse=True, **a)
    again = sv.tree_attention(with_lse=True, **a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = sv.tree_attention(with_lse=True, **a)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            captured = sv.tree_attention(with_lse=True, **a)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for k in ("out", "lse", "status"):
        for r in (again, other, captured):
            assert torch.equal(first[k], r[k]), k


def test_given_outputs_unaligned_queries_and_host_queries():
    c = paged.Case(17, [70], 6, 2, 4, 128, 16, "bf16", True)
    a = c.args()
    out = torch.full_like(a["q"], 7.0)
    got = sv.tree_attention(with_lse=True, out={"out": out}, **a)
    assert got["out"] is out
    store = torch.empty(a["q"].numel() + 1, dtype=torch.bfloat16, device="cuda")
    odd = store[1:].view(a["q"].shape).copy_(a["q"])
    a["q"] = odd
    assert torch.equal(sv.tree_attention(**a)["out"], out)
    a["q"] = c.q
    host = sv.tree_attention(**a)["out"]
    assert host.device.type == "cpu" and torch.equal(host, out.cpu())


def test_refusals():
    c = paged.Case(18, [70, 9], 6, 2, 4, 128, 16, "bf16", True)
    a = c.args()

    def no(**over):
        with pytest.raises(sv.SpecError):
            sv.tree_attention(**{**a, **over})

    no(q=a["q"].float())
    no(q=a["q"][:, :, :7])
    no(q=a["q"][..., :64])
    no(v_cache=a["v_cache"].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3))
    no(k_cache=a["k_cache"][..., ::2], v_cache=a["v_cache"][..., ::2], q=a["q"][..., :64])
    no(page_table=a["page_table"][:1])
    no(page_table=a["page_table"].long())
    no(cache_len=a["cache_len"][:1])
    no(mask=a["mask"][:, :5])
    no(n_nodes=a["n_nodes"][:1])
    no(scale=float("inf"))
    no(scale=float("nan"))
    no(k_cache=a["k_cache"][:, :12], v_cache=a["v_cache"][:, :12])   # page size no power of two
    no(k_cache=a["k_cache"].cpu(), v_cache=a["v_cache"].cpu())
    with pytest.raises(sv.SpecError):                                # head_dim no multiple of 8
        sv.tree_attention(a["q"][..., :12], a["k_cache"][..., :12], a["v_cache"][..., :12], a["page_table"],
                          a["cache_len"])
