"""cache_append_rotary against the definition in 64 bits.

Tolerances. A cosine or sine: the reduced angle is at most pi / 4, rounded once
(2^-24 of it), and the function itself is off by 2 units at the most: below
2^-22, the factor's product included. A result is two products of such and a
sum, below 2^-21 (|a| + |b|) factor, and then rounded to the type by half a step,
2^-8 of it in bf16.
"""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from paged import TD, Case

pytestmark = pytest.mark.gpu


def rotated(x, angle, dim, interleaved, factor):
    """x [n, heads, D] and angle [n, dim / 2], float64; the result and sum |a| + |b| of each element's pair."""
    y, size = x.clone(), x.abs()
    j = torch.arange(dim // 2)
    p, r = (2 * j, 2 * j + 1) if interleaved else (j, j + dim // 2)
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y[..., p], y[..., r] = factor * (x[..., p] * c - x[..., r] * s), factor * (x[..., r] * c + x[..., p] * s)
    size[..., p] = size[..., r] = factor * (x[..., p].abs() + x[..., r].abs())
    return y, size


def angles(rot, pos):
    """2 pi times the fraction of a turn, from the table's integers (exact until the last step)."""
    t = [x % 2 ** 64 for x in rot.turns.tolist()]
    return torch.tensor([[2 * math.pi * (((x * int(p)) % 2 ** 64) / 2.0 ** 64) for x in t] for p in pos],
                        dtype=torch.float64).view(len(pos), len(t))


def run(c, rot, dim, positions=None, depth=None, page_refs=None):
    kc, vc = c.caches()
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(c.B, c.N, c.Hkv, c.D, generator=g).to(TD[c.dtype]) for _ in range(2))
    r = sv.cache_append_rotary(c.q.cuda(), k.cuda(), v.cuda(), kc, vc, torch.from_numpy(c.table).cuda(),
                               torch.from_numpy(c.lens.astype(np.int32)).cuda(), rot,
                               positions=None if positions is None else torch.tensor(positions, dtype=torch.int32).cuda(),
                               depth=None if depth is None else torch.from_numpy(depth).cuda(),
                               n_nodes=torch.from_numpy(c.counts.astype(np.int32)).cuda(), page_refs=page_refs)
    return r, kc.cpu(), vc.cpu(), k, v


def check(c, rot, dim, positions=None, depth=None):
    r, kc, vc, k, v = run(c, rot, dim, positions, depth)
    assert r["status"].tolist() == [0] * c.B
    half = 2.0 ** -8 if c.dtype == "bf16" else 2.0 ** -24
    q = r["q"].double().cpu()
    want_k, want_v = c.k.clone().double(), c.v.clone()
    tol_k = torch.zeros_like(want_k)
    for b in range(c.B):
        n, L = int(c.counts[b]), int(c.lens[b])
        pos0 = L if positions is None else positions[b]
        pos = [pos0 + (i if depth is None else int(depth[b, i])) for i in range(n)]
        a = angles(rot, pos)
        y, size = rotated(c.q[b, :n].double(), a, dim, rot.interleaved, rot.factor)
        assert ((q[b, :n] - y).abs() <= 2.0 ** -21 * size + half * y.abs()).all()
        assert (q[b, n:] == 0).all()
        y, size = rotated(k[b, :n].double(), a, dim, rot.interleaved, rot.factor)
        for i in range(n):
            at = c.table[b, (L + i) // c.ps], (L + i) % c.ps
            want_k[at], tol_k[at], want_v[at] = y[i], 2.0 ** -21 * size[i] + half * y[i].abs(), v[b, i]
    assert ((kc.double() - want_k).abs() <= tol_k).all()   # (what was there before is untouched)
    assert torch.equal(vc, want_v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,dim", [(8, 8), (8, 2), (64, 64), (64, 24), (64, 32), (96, 24), (128, 128), (128, 64), (256, 256),
                                   (80, 70), (256, 2)])
def test_layouts_and_partial_heads(dtype, interleaved, D, dim):
    c = Case(D + dim, [0, 5, 37], 9, 2, 3, D, 16, dtype, counts=[9, 1, 6], layout="wide")
    check(c, sv.rotary(dim, interleaved=interleaved), dim)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,Hkv,G,ps", [(1, 1, 1, 1, 8), (1, 5, 8, 4, 16), (70, 1, 2, 1, 32), (3, 700, 2, 2, 64), (5, 161, 5, 7, 16)])
def test_sizes(dtype, B, N, Hkv, G, ps):
    lens = [(37 * b) % 101 for b in range(B)]
    counts = [N if b % 3 else max(0, N - 1 - b) for b in range(B)]
    c = Case(B + N, lens, N, Hkv, G, 64, ps, dtype, tree=False, counts=counts, layout="hnd")
    check(c, sv.rotary(64, scaling="yarn", scale=4.0, original=128), 64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_and_depths(interleaved):
    """Trees far into a text, to the last position there is."""
    c = Case(3, [4, 0, 20, 7], 12, 2, 2, 64, 16, "f32", counts=[12, 3, 0, 12])
    rng = np.random.default_rng(1)
    depth = rng.integers(0, 8, (4, 12)).astype(np.int32)
    depth[1, 3:] = -1   # (unused nodes: not read)
    depth[2] = -1
    check(c, sv.rotary(64, interleaved=interleaved), 64, [1000003, 2 ** 31 - 9, 0, 131071], depth)
    check(c, sv.rotary(32, interleaved=interleaved, scaling="linear", scale=2.0), 32, [5, 0, 1, 99], None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_data_writes_nothing(dtype):
    c = Case(8, [5, 6, 7, 8, 9, 10, 11], 4, 2, 2, 64, 16, dtype, tree=False)
    c.table[1, 0] = c.P       # no such page
    c.lens[2] = -1
    c.counts[3] = 5
    depth = np.tile(np.arange(4, dtype=np.int32), (7, 1))
    depth[4, 2] = -3
    positions = [0, 1, 2, 3, 4, 2 ** 31 - 3, -1]
    r, kc, vc, k, v = run(c, sv.rotary(64), 64, positions, depth)
    assert r["status"].tolist() == [0] + [sv.SPEC_EDATA] * 6
    assert torch.isfinite(r["q"][0]).all() and torch.isnan(r["q"][1:]).all()
    pages = c.table[0]
    other = [p for p in range(c.P) if p not in pages]
    assert torch.equal(kc[other], c.k[other]) and torch.equal(vc[other], c.v[other])


def test_shared_pages_are_refused_with_counts():
    c = Case(9, [5, 6], 4, 2, 2, 64, 16, "f32", tree=False)
    refs = torch.ones(c.P, dtype=torch.int32, device="cuda")
    refs[c.table[1, 0]] = 2
    r, kc, _, _, _ = run(c, sv.rotary(64), 64, page_refs=refs)
    assert r["status"].tolist() == [0, sv.SPEC_EDATA]
    assert torch.equal(kc[c.table[1, 0]], c.k[c.table[1, 0]])


def test_values_pass_through_what_is_not_finite():
    c = Case(10, [3], 2, 1, 1, 64, 16, "f32", tree=False)
    c.q[0, 0, 0, 0], c.q[0, 1, 0, 63] = math.nan, math.inf
    r, *_ = run(c, sv.rotary(32), 32)
    q = r["q"].cpu()
    assert torch.isnan(q[0, 0, 0, [0, 16]]).all() and torch.isfinite(q[0, 0, 0, 1:16]).all()
    assert q[0, 1, 0, 63] == math.inf and torch.isfinite(q[0, 1, 0, :63]).all()


def test_agrees_with_the_plain_append_at_position_zero():
    """At position 0 nothing turns: the same cache as cache_append, queries as they came."""
    c = Case(11, [21, 2], 5, 2, 2, 128, 16, "bf16", tree=False)
    r, kc, vc, k, v = run(c, sv.rotary(128), 128, [0, 0], np.zeros((2, 5), np.int32))
    k2, v2 = c.caches()
    sv.cache_append(k.cuda(), v.cuda(), k2, v2, torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens.astype(np.int32)).cuda())
    assert torch.equal(kc, k2.cpu()) and torch.equal(vc, v2.cpu()) and torch.equal(r["q"].cpu(), c.q)


def test_streams_graphs_and_arguments():
    c = Case(12, [21, 2], 5, 2, 2, 64, 16, "bf16", tree=False)
    rot = sv.rotary(64)
    kc, vc = c.caches()
    k, v = (torch.randn(2, 5, 2, 64, device="cuda").bfloat16() for _ in range(2))
    q, table, lens = c.q.cuda(), torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens.astype(np.int32)).cuda()
    want = sv.cache_append_rotary(q, k, v, kc, vc, table, lens, rot)["q"]
    after = kc.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sv.cache_append_rotary(q, k, v, kc, vc, table, lens, rot)
    kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["q"], want)
    t = c.table[0]
    assert torch.equal(kc[t[1], 5:10], after[t[1], 5:10])
    # views that start anywhere, lengths of another integer type
    flat = torch.zeros(q.numel() + 1, dtype=q.dtype, device="cuda")
    flat[1:] = q.flatten()
    assert torch.equal(sv.cache_append_rotary(flat[1:].view_as(q), k, v, kc, vc, table, lens.long(), rot)["q"], want)
    for bad in (dict(q=q[:, :4]), dict(q=q.float()), dict(q=q[..., :32]), dict(k=k[:1]), dict(v=v.float()),
                dict(cache_len=lens[:1]), dict(positions=lens[:1]), dict(n_nodes=lens[:1]), dict(depth=lens),
                dict(rotary=sv.rotary(64, device="cpu")), dict(rotary=sv.rotary(66)),
                dict(rotary=rot._replace(factor=math.nan)), dict(rotary=rot._replace(turns=rot.turns.int()))):
        a = dict(q=q, k=k, v=v, k_cache=kc, v_cache=vc, page_table=table, cache_len=lens, rotary=rot)
        a.update(bad)
        with pytest.raises(sv.SpecError):
            sv.cache_append_rotary(**a)
