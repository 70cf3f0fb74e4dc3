"""The paged cache's moves and pages (spec_cache_append, spec_cache_compact,
spec_cache_resize, spec_cache_fork) against their definitions, bit for bit."""

import numpy as np
import pytest
import torch

import paged
import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _same(a, b):
    """Equal bits (NaN included)."""
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    view = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(view), b.view(view))


def _layers(c, layers, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (layers, c.P, c.ps, c.Hkv, c.D)
    return tuple(torch.randn(shape, generator=g).to(paged.TD[c.dtype]) for _ in range(2))


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 8), ("f32", 128), ("f32", 24)])
@pytest.mark.parametrize("N,counts", [(1, None), (9, [9, 4, 0, 1]), (70, [70, 64, 3, 17])])
@pytest.mark.parametrize("ps", [8, 64])
def test_append(dtype, D, N, counts, ps):
    c = paged.Case(20, [0, 7, 64, 130], N, 3, 1, D, ps, dtype, False, counts=counts)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(4, N, 3, D, generator=g).to(paged.TD[dtype]) for _ in range(2))
    kc, vc = c.caches()
    st = sv.cache_append(k.cuda(), v.cuda(), kc, vc, _dev(c.table), _dev(c.lens.astype(np.int32)),
                         n_nodes=None if counts is None else _dev(np.asarray(counts, np.int32)))["status"]
    assert st.tolist() == [0] * 4
    for b in range(4):
        for i in range(int(c.counts[b])):
            t = int(c.lens[b]) + i
            c.k[c.table[b, t // ps], t % ps] = k[b, i]
            c.v[c.table[b, t // ps], t % ps] = v[b, i]
    assert _same(kc, c.k) and _same(vc, c.v)


def test_append_into_other_orders_and_bad_data():
    for layout in ("hnd", "wide"):
        c = paged.Case(21, [5, 40, 17, 3, 9], 6, 2, 1, 64, 16, "bf16", False, layout=layout)
        k, v = (torch.randn(5, 6, 2, 64).bfloat16() for _ in range(2))
        kc, vc = c.caches()
        lens, table = _dev(c.lens.astype(np.int32)), _dev(c.table)
        lens[1] = -3
        table[2, 1] = c.P
        lens[3] = 16 * c.M
        n = torch.tensor([6, 6, 6, 6, 7], dtype=torch.int32)
        st = sv.cache_append(k.cuda(), v.cuda(), kc, vc, table, lens, n_nodes=n)["status"]
        assert st.tolist() == [0, 4, 4, 4, 4]
        for i in range(6):
            t = 5 + i
            c.k[c.table[0, t // 16], t % 16] = k[0, i]
            c.v[c.table[0, t // 16], t % 16] = v[0, i]
        assert _same(kc, c.k) and _same(vc, c.v), layout


@pytest.mark.parametrize("dtype,D,layers", [("bf16", 128, 3), ("f32", 64, 1), ("bf16", 8, 5)])
@pytest.mark.parametrize("W", [1, 2, 8, 33])
def test_compact(dtype, D, layers, W):
    rng = np.random.default_rng(W)
    lens = [0, 1, 15, 16, 33, 70]
    c = paged.Case(22, lens, 60, 2, 1, D, 16, dtype, False)
    k, v = _layers(c, layers, 4)
    acc = np.array([W - 1, 0, (W - 1) // 2, W - 1, W - 1, min(1, W - 1)], np.int32)
    path = np.full((6, W), -1, np.int32)
    for b in range(6):
        path[b, 0] = 0
        path[b, 1:acc[b] + 1] = np.sort(rng.choice(np.arange(1, 60), acc[b], replace=False))
    path[3, :acc[3] + 1] = np.arange(acc[3] + 1)                        # in place already
    if W > 2:
        path[4, :acc[4] + 1] = np.r_[0, 1, np.arange(3, acc[4] + 2)]    # every source is the next one's place
    kd, vd = k.cuda(), v.cuda()
    r = sv.cache_compact(kd, vd, _dev(c.table), _dev(c.lens.astype(np.int32)), _dev(acc), _dev(path))
    assert r["status"].tolist() == [0] * 6
    assert r["cache_len"].tolist() == [l + a + 1 for l, a in zip(lens, acc.tolist())]
    for x in (k, v):
        old = x.clone()
        for b in range(6):
            for i in range(acc[b] + 1):
                s, t = lens[b] + int(path[b, i]), lens[b] + i
                x[:, c.table[b, t // 16], t % 16] = old[:, c.table[b, s // 16], s % 16]
    assert _same(kd, k) and _same(vd, v)


def test_compact_chain_and_bad_data():
    c = paged.Case(23, [10, 20, 30, 40, 50, 60], 8, 2, 1, 64, 16, "bf16", False)
    k, v = _layers(c, 2, 5)
    kd, vd = k.cuda(), v.cuda()
    table, lens = _dev(c.table), _dev(c.lens.astype(np.int32))
    acc = torch.tensor([0, 3, 7, 2, 1, 4], dtype=torch.int32)
    r = sv.cache_compact(kd, vd, table, lens, acc)
    assert r["status"].tolist() == [0] * 6 and r["cache_len"].tolist() == [11, 24, 38, 43, 52, 65]
    path = torch.tensor([[0, 2, 5], [1, 2, 3], [0, 3, 3], [0, 2, -1], [0, 1, 4], [0, 1, 2]], dtype=torch.int32)
    acc = torch.tensor([2, 2, 2, 2, 3, 2], dtype=torch.int32)
    table[5, 3] = -1
    r = sv.cache_compact(kd, vd, table, lens, acc, path)
    assert r["status"].tolist() == [0, 4, 4, 4, 4, 4]
    assert r["cache_len"].tolist() == [13, -1, -1, -1, -1, -1]
    for x in (k, v):
        old = x.clone()
        for i, n in ((1, 2), (2, 5)):
            s, t = 10 + n, 10 + i
            x[:, c.table[0, t // 16], t % 16] = old[:, c.table[0, s // 16], s % 16]
    assert _same(kd, k) and _same(vd, v)
    assert sv.cache_compact(kd, vd, table, lens, torch.full((6,), -1, dtype=torch.int32))["status"].tolist() == [4] * 6


def test_verified_tree_to_compacted_cache():
    """verify_tree's outputs as they come: a data error there (-1) is one here."""
    z = torch.zeros(2, 4, 50, device="cuda")
    z[0, 0, 7] = z[0, 2, 9] = 1.0
    tok = torch.tensor([[1, 5, 7, 9], [1, 2, 3, 4]], dtype=torch.int32)
    par = torch.tensor([[-1, 0, 0, 2], [-1, 0, 3, 0]], dtype=torch.int32)   # second: no breadth-first order
    dep = torch.tensor([[0, 1, 1, 2], [0, 1, 1, 1]], dtype=torch.int32)
    r = sv.verify_tree(z, tok, par, dep, 2)
    c = paged.Case(24, [5, 5], 4, 1, 1, 64, 16, "bf16", False)
    k, v = (x.cuda() for x in _layers(c, 1, 6))
    out = sv.cache_compact(k, v, _dev(c.table), _dev(c.lens.astype(np.int32)), r["accept_len"], r["path_nodes"])
    assert out["cache_len"].tolist() == [8, -1] and out["status"].tolist() == [0, 4]


class Pool:
    def __init__(self, S, M, P, layers=2, ps=16, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.k, self.v = (torch.randn(layers, P, ps, 2, 64, generator=g).bfloat16() for _ in range(2))
        self.table, self.refs = np.full((S, M), -1, np.int32), np.zeros(P, np.int32)
        self.lens, self.ps = np.zeros(S, np.int32), ps
        self.dk, self.dv = self.k.cuda(), self.v.cuda()
        self.dt, self.dr, self.dl = _dev(self.table), _dev(self.refs), _dev(self.lens)

    def resize(self, seqs, tokens):
        want = paged.grow(self.table, self.refs, seqs, tokens, self.ps)
        got = sv.cache_resize(self.dt, self.dr, _dev(np.asarray(seqs, np.int32)), _dev(np.asarray(tokens, np.int32)),
                              self.ps)["status"].tolist()
        assert got == want
        self.same()
        return want

    def fork(self, src, dst):
        want = paged.fork(self.k, self.v, self.table, self.lens, self.refs, src, dst, self.ps)
        got = sv.cache_fork(self.dk, self.dv, self.dt, self.dl, self.dr, _dev(np.asarray(src, np.int32)),
                            _dev(np.asarray(dst, np.int32)))["status"].tolist()
        assert got == want
        self.same()
        return want

    def set_len(self, s, n):
        self.lens[s] = n
        self.dl[s] = n

    def same(self):
        np.testing.assert_array_equal(self.dt.cpu().numpy(), self.table)
        np.testing.assert_array_equal(self.dr.cpu().numpy(), self.refs)
        np.testing.assert_array_equal(self.dl.cpu().numpy(), self.lens)
        assert _same(self.dk, self.k) and _same(self.dv, self.v)


def test_grow_shrink_free():
    p = Pool(6, 8, 20)
    p.resize([0, 1, 2], [1, 16, 17])
    p.resize([2, 0, 1], [100, 0, 16])          # what 0 gives back, 2 takes
    p.resize([5, 3], [128, 0])
    p.resize([0, 1, 2, 3, 4, 5], [0] * 6)
    assert (p.refs == 0).all()


def test_errors_and_shortage():
    p = Pool(5, 6, 10)
    assert p.resize([0, 7, -1, 1, 2], [40, 5, 5, -1, 97]) == [0, 4, 4, 4, 4]
    assert p.resize([1, 2, 3, 4], [64, 64, 16, 0]) == [0, 6, 6, 0]      # 7 free: 4 + 4 do not fit, nor does what follows
    assert p.resize([2, 0], [48, 16]) == [0, 0]
    p.table[2, 0] = p.dt[2, 0] = 10                                      # no such page
    assert p.resize([2, 3], [0, 16]) == [4, 0]


def test_all_sequences_without_a_list():
    p = Pool(40, 4, 160)
    tok = np.arange(40, dtype=np.int32)
    want = paged.grow(p.table, p.refs, range(40), tok, 16)
    assert sv.cache_resize(p.dt, p.dr, None, _dev(tok), 16)["status"].tolist() == want
    p.same()


def test_random_history():
    """Pages after many calls: as the definition has them, every count the number of entries."""
    rng = np.random.default_rng(3)
    p = Pool(24, 10, 90, layers=1)
    for step in range(30):
        free_rows = [s for s in range(24) if p.table[s, 0] == -1]
        used = [s for s in range(24) if p.table[s, 0] != -1]
        if step % 3 == 2 and used and free_rows:
            dst = list(rng.permutation(free_rows)[:rng.integers(1, len(free_rows) + 1)])
            p.fork([int(rng.choice(used)) for _ in dst], [int(d) for d in dst])
        else:
            seqs = [int(s) for s in rng.permutation(24)[:rng.integers(1, 12)]]
            tokens = [int(rng.choice([0, 0, rng.integers(1, 161)])) for _ in seqs]
            st = p.resize(seqs, tokens)
            for s, t, r in zip(seqs, tokens, st):
                if r == 0:
                    p.set_len(s, t)
        held = p.table[p.table >= 0]
        np.testing.assert_array_equal(np.bincount(held, minlength=90), p.refs)


@pytest.mark.parametrize("pages", [4095, 4097, 8200, 32771, 70000, 131072])
@pytest.mark.parametrize("shift", [0, 1])
def test_free_pages_anywhere_in_a_pool(pages, shift):
    """The lowest free numbers, wherever they lie: windows and stretches without any, the last page, odd addresses."""
    rng = np.random.default_rng(pages + shift)
    free = np.unique(np.concatenate([rng.integers(0, pages, 40), rng.integers(max(0, pages - 50), pages, 9), [pages - 1],
                                     np.arange(pages // 2, min(pages, pages // 2 + 30))]))
    refs = np.ones(pages, np.int32)
    refs[free] = 0
    store = torch.ones(pages + 1, dtype=torch.int32, device="cuda")
    dr = store[shift:shift + pages].copy_(torch.from_numpy(refs))
    for tokens in ([16 * 20, 0, 5, 16 * 30], [16 * len(free), 0, 0, 0], [0, 0, 0, 16 * len(free) + 1], [16, 16, 16 * 39, 16]):
        table = np.full((4, len(free) + 2), -1, np.int32)
        dt, r = _dev(table), refs.copy()
        dr.copy_(torch.from_numpy(refs))
        want = paged.grow(table, r, [0, 1, 2, 3], tokens, 16)
        got = sv.cache_resize(dt, dr, None, torch.tensor(tokens, dtype=torch.int32), 16)["status"].tolist()
        assert got == want
        np.testing.assert_array_equal(dt.cpu().numpy(), table)
        np.testing.assert_array_equal(dr.cpu().numpy(), r)


def test_large_pool_takes_the_last_pages():
    p = Pool(3, 300, 70001, layers=1, ps=8)
    p.refs[:69000] = 1
    p.refs[69500] = 2
    p.dr.copy_(_dev(p.refs))
    assert p.resize([2, 0, 1], [2400, 2400, 2400]) == [0, 0, 0]
    assert p.resize([1, 2], [0, 2300]) == [0, 0]


@pytest.mark.parametrize("ps", [8, 32, 256])
def test_fork(ps):
    p = Pool(12, 6, 60, layers=3, ps=ps)
    p.resize([0, 1, 2, 3], [5 * ps + 3, 2 * ps, 1, 0])
    for s, n in ((0, 5 * ps + 3), (1, 2 * ps), (2, 1)):
        p.set_len(s, n)
    assert p.fork([0, 0, 1, 2, 3], [4, 11, 5, 6, 7]) == [0] * 5
    assert p.fork([4, 0], [8, 9]) == [0, 0]
    p.resize([0, 4], [0, 0])                                            # the shared pages stay
    assert p.fork([9, 0, 1, 1, 12, 2], [10, 3, 1, 8, 3, -1]) == [0, 4, 4, 4, 4, 4]


def test_fork_without_pages_left():
    p = Pool(8, 4, 6)
    p.resize([0, 1], [40, 16])
    p.set_len(0, 40)
    p.set_len(1, 16)
    assert p.fork([0, 0, 1, 0], [2, 3, 4, 5]) == [0, 0, 0, 6]


def test_float32_and_strided_caches_fork():
    p = Pool(4, 3, 8)
    p.resize([0], [21])
    p.set_len(0, 21)
    for make in (lambda x: x.float().cuda(),
                 lambda x: x.permute(1, 0, 3, 2, 4).contiguous().cuda().permute(1, 0, 3, 2, 4)):
        k, v = make(p.k), make(p.v)
        t, l, r = p.dt.clone(), p.dl.clone(), p.dr.clone()
        assert sv.cache_fork(k, v, t, l, r, torch.tensor([0]), torch.tensor([3]))["status"].tolist() == [0]
        assert t[3].tolist()[:2] == [0, 2] and l[3] == 21
        assert torch.equal(k[:, 2, :5], k[:, 1, :5]) and torch.equal(v[:, 2, :5], v[:, 1, :5])
        assert torch.equal(k[:, 2, 5:].cpu(), p.k[:, 2, 5:].to(k.dtype))


def test_refusals():
    p = Pool(4, 3, 8)
    one, two = torch.tensor([0]), torch.tensor([0, 1])
    for bad in (lambda: sv.cache_resize(p.dt, p.dr, one, two, 16), lambda: sv.cache_resize(p.dt, p.dr, one, one, 12),
                lambda: sv.cache_resize(p.dt.cpu(), p.dr.cpu(), one, one, 16),
                lambda: sv.cache_resize(p.dt, p.dr, None, torch.zeros(5), 16),
                lambda: sv.cache_resize(p.dt, p.dr.long(), one, one, 16),
                lambda: sv.cache_fork(p.dk, p.dv, p.dt, p.dl, p.dr[:5], one, one),
                lambda: sv.cache_fork(p.dk, p.dv, p.dt, p.dl[:3], p.dr, one, one),
                lambda: sv.cache_fork(p.dk[0], p.dv[0], p.dt, p.dl, p.dr, one, one),
                lambda: sv.cache_fork(p.dk, p.dv, p.dt, p.dl, p.dr, one, two),
                lambda: sv.cache_compact(p.dk, p.dv, p.dt, p.dl, p.dl[:2]),
                lambda: sv.cache_compact(p.dk, p.dv, p.dt, p.dl, p.dl, p.dt[:2]),
                lambda: sv.cache_append(p.dk[0, :4, :1], p.dv[0, :4, :1], p.dk[0], p.dv[0, :, :8], p.dt, p.dl),
                lambda: sv.cache_append(p.dk[0, :4, :1].float(), p.dv[0, :4, :1].float(), p.dk[0], p.dv[0], p.dt, p.dl),
                lambda: sv.cache_append(p.dk[0, :3, :1], p.dv[0, :3, :1], p.dk[0], p.dv[0], p.dt, p.dl)):
        with pytest.raises(sv.SpecError):
            bad()
    p.same()
