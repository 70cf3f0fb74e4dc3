"""cache_weigh against the definition in 64 bits.

Tolerances. A score: a dot product of D terms, off by (D + 8) 2^-23 of the sum of
their sizes at the most (the factor and the exponent's rounding included, and the
tensor cores' sums, which may cut off a bit more than they round); the log-sum's
product 2^-23 of it; the exponential 2^-22. A position's sum of R terms of one
sign is off by R 2^-24, and its addition to what was there by 2^-24 of the result.
"""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from paged import Case

pytestmark = pytest.mark.gpu


def paths(rng, B, N, W, accept):
    p = np.full((B, W), -1, np.int32)
    for b in range(B):
        a = int(accept[b])
        if a >= 0:
            p[b, 0] = 0
            p[b, 1:a + 1] = np.sort(rng.choice(np.arange(1, N), size=a, replace=False))
    return p


class Weigh:
    def __init__(self, seed, lens, N, Hkv, G, D, ps, dtype, accept=None, path=None, capacity=None, layout="nhd", q_scale=1.5,
                 scale=None):
        self.n = np.full(len(lens), N) if accept is None else np.asarray(accept) + 1
        self.c = c = Case(seed, lens, N, Hkv, G, D, ps, dtype, tree=False, counts=self.n, layout=layout, garbage=math.nan,
                          q_scale=q_scale)
        self.accept, self.path = accept, path
        self.scale = D ** -0.5 if scale is None else scale
        g = torch.Generator().manual_seed(seed)
        self.T = c.M * ps if capacity is None else capacity
        self.w = torch.rand(c.B, Hkv, self.T, generator=g)
        self.lse = torch.full((c.B, N, Hkv * G), math.nan)   # (of rows that are not weighed: not read)
        self.want, self.tol = self.w.double(), torch.zeros(c.B, Hkv, self.T, dtype=torch.float64)
        for b in range(c.B):
            n, L = int(self.n[b]), int(lens[b])
            if n <= 0:
                continue
            nodes = np.arange(n) if path is None else path[b, :n]
            k = c.rows(b, c.k)                                                        # [L + n, Hkv, D]
            q = c.q[b, torch.from_numpy(np.asarray(nodes)).long()].double().view(n, Hkv, G, D)
            s = torch.einsum("nhgd,thd->nhgt", q, k) * self.scale
            size = torch.einsum("nhgd,thd->nhgt", q.abs(), k.abs()) * abs(self.scale)
            see = torch.arange(L + n)[None] <= L + torch.arange(n)[:, None]
            s = s.masked_fill(~see[:, None, None], -math.inf)
            z = torch.logsumexp(s, -1).float()
            self.lse[b, torch.from_numpy(np.asarray(nodes)).long()] = z.reshape(n, -1)
            p = torch.exp(s - z.double()[..., None])
            rel = (D + 8) * 2.0 ** -23 * size + 2.0 ** -23 * z.abs().double()[..., None] + 2.0 ** -22 + n * G * 2.0 ** -24
            self.want[b, :, :L + n] += p.sum((0, 2))
            self.tol[b, :, :L + n] = (p * rel).sum((0, 2)) + 2.0 ** -23 * self.want[b, :, :L + n] + 1e-37

    def args(self):
        c = self.c
        i32 = lambda x: None if x is None else torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()
        return dict(q=c.q.cuda(), lse=self.lse.cuda(), k_cache=c.caches()[0], page_table=torch.from_numpy(c.table).cuda(),
                    cache_len=i32(c.lens), weights=self.w.cuda(), accept_len=i32(self.accept), path_nodes=i32(self.path),
                    scale=self.scale)

    def check(self, status=None, **kw):
        a = {**self.args(), **kw}
        r = sv.cache_weigh(**a)
        assert r["status"].tolist() == (status or [0] * self.c.B)
        off = (a["weights"].double().cpu() - self.want).abs()
        assert (off <= self.tol).all(), float((off / self.tol.clamp(min=1e-37)).max())
        return a["weights"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 64, 96, 128, 256])
@pytest.mark.parametrize("lens,N,Hkv,G,ps", [
    ([0], 1, 1, 1, 8), ([1, 63, 64, 65], 1, 2, 4, 16), ([127, 128, 129, 0, 300], 5, 2, 1, 32), ([17, 600], 3, 1, 7, 64),
    ([250], 40, 2, 4, 128), ([5, 33, 129], 61, 1, 8, 16)])
def test_chains_and_tokens(dtype, D, lens, N, Hkv, G, ps):
    Weigh(D + N, lens, N, Hkv, G, D, ps, dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,W,Hkv,G,ps", [(64, 7, 2, 8, 16), (30, 17, 3, 3, 32), (200, 130, 1, 2, 64), (5, 1, 2, 1, 8)])
def test_accepted_paths(dtype, D, N, W, Hkv, G, ps):
    rng = np.random.default_rng(N)
    lens = [0, 5, 130, 700, 64, 257]
    accept = np.minimum(rng.integers(0, W, 6), N - 1)
    accept[2] = -1      # (nothing was accepted: nothing is added)
    Weigh(N, lens, N, Hkv, G, D, ps, dtype, accept, paths(rng, 6, N, W, accept)).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["hnd", "wide"])
def test_accepted_chains_and_layouts(dtype, layout):
    Weigh(5, [3, 77, 400], 8, 2, 4, 64, 16, dtype, accept=[7, 0, 3], layout=layout).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(dtype):
    """Prompt chunks: more rows than any tile holds."""
    Weigh(6, [0, 200], 300, 1, 4, 64, 16, dtype).check()
    Weigh(7, [500], 1000, 1, 1, 128, 64, dtype).check()
    Weigh(8, [100], 3, 1, 128, 64, 16, dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(dtype):
    Weigh(9, [(61 * b) % 300 for b in range(300)], 2, 1, 2, 64, 16, dtype, accept=[b % 3 - 1 for b in range(300)]).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(dtype, scale):
    Weigh(10, [70, 9], 4, 2, 2, 64, 16, dtype, scale=scale, q_scale=0.5).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("capacity", [136, 137, 500])
def test_capacities(dtype, capacity):
    """Weights of any capacity from the last position on; positions past the end are left as they were."""
    Weigh(11, [128, 3, 60], 8, 2, 2, 64, 16, dtype, capacity=capacity).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(dtype):
    """A log-sum of -inf (a row that sees nothing), NaN and +inf."""
    w = Weigh(12, [40, 41, 42, 43], 2, 1, 2, 64, 16, dtype)
    a = w.args()
    a["lse"][0] = -math.inf
    a["lse"][1, 0] = -math.inf
    a["lse"][2] = math.inf
    a["lse"][3, 1, 1] = math.nan
    before = a["weights"].clone()
    assert sv.cache_weigh(**a)["status"].tolist() == [0] * 4
    assert torch.equal(a["weights"][0], before[0]) and torch.equal(a["weights"][2], before[2])
    assert torch.isfinite(a["weights"][1]).all() and (a["weights"][1, :, :43] >= before[1, :, :43]).all()
    assert torch.isnan(a["weights"][3, :, :45]).all() and torch.equal(a["weights"][3, :, 45:], before[3, :, 45:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_data(dtype):
    N, B = 6, 8
    accept = np.array([2, 6, -2, 3, 2, 2, 2, 1])
    good = np.clip(accept, 0, 5)
    path = np.tile(np.arange(6, dtype=np.int32), (B, 1))
    lens = [50] * B
    w = Weigh(13, lens, N, 1, 2, 64, 16, dtype, good, path)
    a = w.args()
    a["accept_len"] = torch.from_numpy(accept.astype(np.int32)).cuda()
    a["path_nodes"][3, 1] = N
    a["path_nodes"][4, 2] = -1
    a["cache_len"][5] = -1
    a["page_table"][6, 1] = -1
    a["cache_len"][7] = 10000
    before = a["weights"].clone()
    r = sv.cache_weigh(**a)
    assert r["status"].tolist() == [0] + [sv.SPEC_EDATA] * 7
    got = a["weights"]
    for b in (1, 2, 3, 4, 5, 7):
        assert torch.equal(got[b], before[b]), b
    off = (got[:1].double().cpu() - w.want[:1]).abs()
    assert (off <= w.tol[:1]).all()
    assert torch.equal(got[6, :, 16:32], before[6, :, 16:32])
    # a capacity that a sequence's positions pass
    a = w.args()
    a["weights"] = a["weights"][..., :52].contiguous()
    before = a["weights"].clone()
    r = sv.cache_weigh(**a)
    assert r["status"].tolist() == [0 if 50 + g + 1 <= 52 else sv.SPEC_EDATA for g in good]
    assert torch.equal(a["weights"][1], before[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sums_repeat(dtype):
    w = Weigh(14, [1000, 3, 500, 77], 9, 2, 4, 128, 16, dtype)
    assert torch.equal(w.check(), w.check())


def test_sums_to_the_rows():
    """Added up over the positions, a head's weights are its rows' number."""
    c = Case(15, [333, 20], 5, 2, 4, 128, 16, "bf16", tree=False)
    a = c.args()
    o = sv.tree_attention(a["q"], a["k_cache"], a["v_cache"], a["page_table"], a["cache_len"], with_lse=True)
    w = torch.zeros(2, 2, c.M * 16, device="cuda")
    sv.cache_weigh(a["q"], o["lse"], a["k_cache"], a["page_table"], a["cache_len"], w)
    assert (w.sum(-1) - 20).abs().max() < 20 * 2.0 ** -12


def test_streams_graphs_and_arguments():
    w = Weigh(16, [100, 9], 4, 2, 2, 64, 16, "bf16")
    a = w.args()
    start = a["weights"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.cache_weigh(**a)
    a["weights"].copy_(start)
    g.replay()
    torch.cuda.synchronize()
    assert ((a["weights"].double().cpu() - w.want).abs() <= w.tol).all()
    s = torch.cuda.Stream()
    a["weights"].copy_(start)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sv.cache_weigh(**a)
    s.synchronize()
    assert ((a["weights"].double().cpu() - w.want).abs() <= w.tol).all()
    q = a["q"]
    for bad in (dict(q=q.float()), dict(q=q[:, :, :3]), dict(q=q[:1]), dict(lse=a["lse"][:, :3]), dict(weights=start.double()),
                dict(weights=start[:, :1]), dict(weights=start[..., ::2]), dict(weights=start.cpu()), dict(cache_len=a["cache_len"][:1]),
                dict(path_nodes=torch.zeros(2, 2, dtype=torch.int32, device="cuda")), dict(accept_len=a["cache_len"][:1]),
                dict(scale=math.nan), dict(scale=math.inf)):
        with pytest.raises(sv.SpecError):
            sv.cache_weigh(**{**a, **bad})


def test_debug_build_agrees():
    w = Weigh(17, [100, 9], 4, 2, 2, 64, 16, "f32")
    x = w.check()
    with sv.use_library(sv.DEBUG_LIB_PATH):
        assert torch.equal(w.check(), x)
        assert sv.load_library().spec_debug_failures(None) == 0
