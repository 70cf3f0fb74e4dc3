"""cache_evict against a plain implementation: what is kept, in which order, is
equal; what moves keeps its bits."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


class Cache:
    def __init__(self, seed, lens, layers, H, D, ps, dtype="bf16", capacity=None, layout="nhd", kind="heavy"):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.layers, self.H, self.D, self.ps = np.asarray(lens, np.int64), layers, H, D, ps
        B = len(lens)
        need = -(-self.lens // ps)
        self.M, self.P = int(max(1, need.max())), int(need.sum()) + 2
        order = rng.permutation(self.P)[:int(need.sum())]
        table = np.full((B, self.M), -1, np.int32)
        table[np.arange(self.M)[None] < need[:, None]] = order
        self.table = torch.from_numpy(table).cuda()
        shape = (layers, self.P, ps, H, D)
        if layout == "hnd":
            make = lambda: torch.randn(layers, self.P, H, ps, D, generator=g, device="cuda").to(TD[dtype]).transpose(2, 3)
        elif layout == "wide":
            make = lambda: torch.randn(layers, self.P, ps, H + 1, D + 16, generator=g, device="cuda").to(TD[dtype])[..., :H, :D]
        else:
            make = lambda: torch.randn(shape, generator=g, device="cuda").to(TD[dtype])
        self.k, self.v = make(), make()
        self.T = self.M * ps if capacity is None else capacity
        w = torch.randn(layers, B, H, self.T, generator=g, device="cuda").mul(2).exp()
        if kind == "ties":
            w = w.round()
        elif kind == "equal":
            w = torch.ones_like(w)
        elif kind == "odd":
            r = torch.rand(w.shape, generator=g, device="cuda")
            w[r < 0.05], w[(r > 0.05) & (r < 0.1)], w[(r > 0.1) & (r < 0.3)] = math.nan, math.inf, 0.0
            w[(r > 0.3) & (r < 0.4)], w[r > 0.95] = -0.0, -1.0
            w[(r > 0.4) & (r < 0.45)] = -math.nan
        self.w = w
        self.len = torch.from_numpy(self.lens.astype(np.int32)).cuda()

    def expected(self, budget, sink, recent, skip=()):
        k, v, w, new = self.k.cpu().clone(), self.v.cpu().clone(), self.w.cpu().clone(), []
        table = self.table.cpu().numpy()
        for b, L in enumerate(self.lens):
            L, keep = int(L), int(budget[b])
            if b in skip:
                new.append(-1)
                continue
            new.append(min(L, keep))
            if L <= keep:
                continue
            at = lambda t: (table[b, t // self.ps], t % self.ps)
            for y in range(self.layers):
                for h in range(self.H):
                    x = self.w[y, b, h, :L].double().cpu().numpy()
                    mid = np.arange(sink, L - recent)
                    xm = np.where(np.isnan(x[mid]), np.inf, x[mid])
                    top = np.isnan(x[mid])
                    order = np.lexsort((mid, -xm, ~top))[:keep - sink - recent]
                    kept = np.sort(np.concatenate([np.arange(sink), mid[order], np.arange(L - recent, L)]))
                    p, s = at(kept)
                    q, r = at(np.arange(keep))
                    k[y, q, r, h], v[y, q, r, h] = self.k[y].cpu()[p, s, h], self.v[y].cpu()[p, s, h]
                    w[y, b, h, :keep] = self.w[y, b, h].cpu()[kept]
                    w[y, b, h, keep:L] = 0.0
        return k, v, w, new

    def check(self, budget, sink=0, recent=0, refs=None, skip=()):
        B = len(self.lens)
        budget = np.broadcast_to(np.asarray(budget, np.int32), (B,))
        k, v, w, new = self.expected(budget, sink, recent, skip)
        r = sv.cache_evict(self.k, self.v, self.table, self.len, self.w, torch.from_numpy(budget.copy()).cuda(), sink, recent,
                           page_refs=refs)
        assert r["status"].tolist() == [sv.SPEC_EDATA if b in skip else 0 for b in range(B)]
        assert r["cache_len"].tolist() == new
        bits = lambda x: x.cpu().contiguous().view(torch.int32 if x.element_size() == 4 else torch.int16)
        assert torch.equal(bits(self.w), bits(w))
        assert torch.equal(bits(self.k), bits(k)) and torch.equal(bits(self.v), bits(v))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "odd"])
@pytest.mark.parametrize("lens,layers,H,D,ps,budget,sink,recent", [
    ([10], 1, 1, 8, 8, 3, 0, 0), ([10, 0, 1, 9], 2, 3, 64, 16, 7, 2, 3), ([100, 33, 64], 2, 2, 128, 32, 32, 4, 28),
    ([300, 299, 17, 301], 1, 5, 96, 16, [200, 299, 0, 300], 0, 0), ([700], 3, 2, 256, 64, 33, 1, 0),
    ([513, 600], 2, 1, 80, 256, 512, 0, 512)])
def test_against_a_plain_implementation(dtype, kind, lens, layers, H, D, ps, budget, sink, recent):
    Cache(len(lens) + D, lens, layers, H, D, ps, dtype, kind=kind).check(budget, sink, recent)


@pytest.mark.parametrize("kind", ["heavy", "ties", "odd"])
@pytest.mark.parametrize("L", [4095, 4096, 4097, 8193, 20001])
def test_long_sequences(kind, L):
    """Up to and past what a block's registers hold, and weights that begin off 16 bytes."""
    Cache(L, [L, 50], 1, 2, 8, 256, "bf16", kind=kind).check(L // 2, 4, 100)
    Cache(L, [L], 1, 3, 8, 256, "bf16", kind=kind, capacity=L + 1).check(L - 1, 0, 1)


@pytest.mark.parametrize("layout", ["hnd", "wide"])
def test_layouts(layout):
    Cache(2, [150, 90], 3, 2, 64, 16, "bf16", layout=layout).check(70, 3, 20)


def test_budgets_that_keep_everything_or_nothing():
    c = Cache(3, [40, 41, 5], 2, 2, 64, 16)
    c.check([40, 41, 100])
    c.check([0, 41, 0])
    c = Cache(4, [40, 41, 5], 2, 2, 64, 16)
    c.check(8, 8, 0)
    c = Cache(4, [40, 41, 5], 2, 2, 64, 16)
    c.check(8, 0, 8)


def test_evicting_again():
    """The shortened cache is a cache like any other."""
    c = Cache(5, [200, 150], 2, 2, 64, 16)
    c.check(100, 2, 10)
    c.lens = np.minimum(c.lens, 100)
    c.len = torch.from_numpy(c.lens.astype(np.int32)).cuda()
    c.check(60, 2, 10)


def test_bad_data_moves_nothing():
    lens = [100] * 6
    c = Cache(6, lens, 2, 2, 64, 16)
    c.len[1] = -1
    c.len[2] = 10000
    c.table[3, 6] = c.P
    c.table[4, 0] = -1
    budget = np.array([60, 60, 60, 60, 60, 9])
    k, v, w, new = c.expected(budget, 4, 6, skip=(1, 2, 3, 4, 5))
    r = sv.cache_evict(c.k, c.v, c.table, c.len, c.w, torch.from_numpy(budget.astype(np.int32)).cuda(), 4, 6)
    assert r["status"].tolist() == [0] + [sv.SPEC_EDATA] * 5 and r["cache_len"].tolist() == [60] + [-1] * 5
    assert torch.equal(c.k.cpu(), k) and torch.equal(c.v.cpu(), v) and torch.equal(c.w.cpu(), w)
    # weights of fewer positions than a sequence has
    c = Cache(7, [100, 40], 1, 2, 64, 16, capacity=99)
    before = c.w.clone()
    r = sv.cache_evict(c.k, c.v, c.table, c.len, c.w, 50)
    assert r["status"].tolist() == [sv.SPEC_EDATA, 0] and torch.equal(before, c.w)


def test_shared_pages_are_refused_with_counts():
    c = Cache(8, [100, 100, 30], 1, 2, 64, 16)
    refs = torch.ones(c.P, dtype=torch.int32, device="cuda")
    refs[c.table[0, 1]] = 2          # a page that would be written
    refs[c.table[1, 0]] = 2          # the sinks' page alone
    refs[c.table[1, 5]] = 2          # a page behind the budget
    refs[c.table[2, 0]] = 2          # a sequence that stays as it is
    c.check(50, 16, 4, refs, skip=(0,))


def test_streams_graphs_and_arguments():
    c, d = Cache(9, [200, 60], 2, 2, 64, 16), Cache(9, [200, 60], 2, 2, 64, 16)
    k, v, w, new = d.expected(np.array([50, 50]), 2, 8)
    start = [x.clone() for x in (c.k, c.v, c.w)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = sv.cache_evict(c.k, c.v, c.table, c.len, c.w, 50, 2, 8)
    s.synchronize()
    assert r["cache_len"].tolist() == new and torch.equal(c.k.cpu(), k) and torch.equal(c.w.cpu(), w)
    budget = torch.tensor([50, 50], dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = sv.cache_evict(c.k, c.v, c.table, c.len, c.w, budget, 2, 8)
    for _ in range(2):
        for x, y in zip((c.k, c.v, c.w), start):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert r["cache_len"].tolist() == new and torch.equal(c.k.cpu(), k) and torch.equal(c.v.cpu(), v)
        assert torch.equal(c.w.cpu(), w)
    a = dict(k_cache=c.k, v_cache=c.v, page_table=c.table, cache_len=c.len, weights=c.w, budget=budget)
    for bad in (dict(weights=c.w[0]), dict(weights=c.w.half()), dict(weights=c.w[:, :1]), dict(weights=c.w.transpose(0, 1)),
                dict(cache_len=c.len[:1]), dict(budget=budget[:1]), dict(sink=-1), dict(recent=-1), dict(k_cache=c.k[0]),
                dict(page_refs=budget)):
        with pytest.raises(sv.SpecError):
            sv.cache_evict(**{**a, **bad})


def test_debug_build_agrees():
    c, d = Cache(10, [200, 60], 2, 2, 64, 16), Cache(10, [200, 60], 2, 2, 64, 16)
    c.check(50, 2, 8)
    with sv.use_library(sv.DEBUG_LIB_PATH):
        d.check(50, 2, 8)
        assert sv.load_library().spec_debug_failures(None) == 0


@pytest.mark.parametrize("dtype,D,page_size", [("bf16", 128, 32), ("f32", 64, 16), ("bf16", 64, 128), ("bf16", 8, 256)])
def test_many_long_lists(dtype, D, page_size):
    """Lists of many batches in all blocks at once, several times: warps that are behind
    must find their batch's places as they were."""
    layers, H, keep, sink, recent = 6, 8, 1300, 4, 300
    lens = [3000 - 37 * b for b in range(8)]
    for seed in range(4):
        c = Cache(seed, lens, layers, H, D, page_size, dtype)
        B, T = len(lens), c.T
        place = torch.arange(T, device="cuda")
        order = c.w.clone()
        order[..., :sink] = math.inf
        for b, L in enumerate(lens):
            order[:, b, :, L - recent:L] = math.inf
            order[:, b, :, L:] = -math.inf
        kept = torch.sort(order, dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values   # [y, b, h, keep]
        page = c.table.long()[None, :, None].expand(layers, B, H, -1)
        y, h = torch.arange(layers, device="cuda")[:, None, None, None], torch.arange(H, device="cuda")[None, None, :, None]
        frm = page.gather(-1, kept // page_size) * page_size + kept % page_size
        to = page.gather(-1, (place[:keep] // page_size).expand_as(kept)) * page_size + place[:keep] % page_size
        want = []
        for cache in (c.k, c.v):
            flat = cache.clone().view(layers, -1, H, D)
            flat[y, to, h] = flat[y, frm, h]
            want.append(flat.view_as(cache))
        w = c.w.gather(-1, kept)
        r = sv.cache_evict(c.k, c.v, c.table, c.len, c.w, keep, sink, recent)
        assert r["cache_len"].tolist() == [keep] * B
        assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1]) and torch.equal(c.w[..., :keep], w)
