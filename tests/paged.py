"""Paged caches for the tests, and the definitions of what the cache operators
compute, in 64 bits and plain Python, one sequence at a time."""

import math

import numpy as np
import torch

TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def tree_mask(rng, n, N):
    """A random breadth-first tree's ancestor mask [N, N] over its first n nodes."""
    m = np.zeros((N, N), np.uint8)
    parent = [-1] * n
    for i in range(n):
        if i:
            parent[i] = int(rng.integers(max(parent[i - 1], 0, i - 5), i))
            m[i] = m[parent[i]]
        m[i, i] = 1
    return m


class Case:
    """Random inputs of one attention call, on the CPU, with the page table in a
    random page order. `garbage` fills what no node may see."""

    def __init__(self, seed, lens, N, Hkv, G, D, page_size, dtype="bf16", tree=True, counts=None, layout="nhd",
                 garbage=None, q_scale=1.5, spare=2):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.B, self.N, self.Hkv, self.G, self.D, self.ps, self.dtype = len(lens), N, Hkv, G, D, page_size, dtype
        self.lens = np.asarray(lens, np.int64)
        self.counts = np.full(self.B, N) if counts is None else np.asarray(counts)
        need = -(-(self.lens + self.counts) // page_size)
        self.M = int(max(1, need.max()))
        self.P = int(need.sum()) + spare
        order = rng.permutation(self.P)[:int(need.sum())]
        self.table = np.full((self.B, self.M), -1, np.int32)
        self.table[np.arange(self.M)[None, :] < need[:, None]] = order
        td = TD[dtype]
        shape = (self.P, page_size, Hkv, D)
        make = lambda: (torch.randn(shape, generator=g) if garbage is None else torch.full(shape, garbage)).to(td)
        self.k, self.v = make(), make()
        if garbage is not None:
            for b in range(self.B):
                for t in range(int(self.lens[b] + self.counts[b])):
                    p, s = self.table[b, t // page_size], t % page_size
                    self.k[p, s] = torch.randn(Hkv, D, generator=g).to(td)
                    self.v[p, s] = torch.randn(Hkv, D, generator=g).to(td)
        self.q = (q_scale * torch.randn(self.B, N, Hkv * G, D, generator=g)).to(td)
        self.mask = np.stack([tree_mask(rng, int(c), N) for c in self.counts]) if tree else None
        self.scale = D ** -0.5
        self.layout = layout

    def caches(self):
        """Device caches in the case's memory layout, all seen as [pages, page_size, heads, D]."""
        if self.layout == "nhd":
            return self.k.cuda(), self.v.cuda()
        if self.layout == "hnd":
            f = lambda x: x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
        else:  # one tensor for both, rows apart by more than their length
            def f(x):
                wide = torch.full((self.P, self.ps, self.Hkv + 1, self.D + 16), float("nan"), dtype=x.dtype, device="cuda")
                wide[:, :, :self.Hkv, :self.D] = x.cuda()
                return wide[:, :, :self.Hkv, :self.D]
        return f(self.k), f(self.v)

    def args(self):
        k, v = self.caches()
        return dict(q=self.q.cuda(), k_cache=k, v_cache=v, page_table=torch.from_numpy(self.table).cuda(),
                    cache_len=torch.from_numpy(self.lens.astype(np.int32)).cuda(),
                    mask=None if self.mask is None else torch.from_numpy(self.mask).cuda(),
                    n_nodes=torch.from_numpy(self.counts.astype(np.int32)).cuda(), scale=self.scale)

    def rows(self, b, cache):
        """Positions 0 .. L + n - 1 of sequence b as float64 [T, heads, D]."""
        T = int(self.lens[b] + self.counts[b])
        at = [(self.table[b, t // self.ps], t % self.ps) for t in range(T)]
        if not at:
            return torch.zeros(0, self.Hkv, self.D, dtype=torch.float64)
        p, s = (torch.tensor(x, dtype=torch.long) for x in zip(*at))
        return cache[p, s].double()

    def expected(self):
        """out, lse, and the bounds that |computed - out| and |computed - lse| have to keep.

        Scores: a dot product of D fp32 terms is off by at most (D + 8) 2^-24 of
        the sum of their sizes (the factor scale * log2(e) and the
        exponential's argument included); a weight is then off by that
        (relative), by the exponential's 2^-22 and, in bf16, by 2^-9 for its
        rounding before the product with v; sums of T fp32 terms of one sign
        are off by at most T 2^-24; bf16 outputs are rounded to 2^-9.
        """
        B, N, H, G, D = self.B, self.N, self.Hkv, self.G, self.D
        out = torch.zeros(B, N, H * G, D, dtype=torch.float64)
        lse = torch.full((B, N, H * G), -math.inf, dtype=torch.float64)
        tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
        half = 2.0 ** -9 if self.dtype == "bf16" else 0.0
        for b in range(B):
            L, n = int(self.lens[b]), int(self.counts[b])
            if n == 0:
                continue
            k, v = self.rows(b, self.k), self.rows(b, self.v)
            see = torch.ones(n, L + n, dtype=torch.bool)
            see[:, L:] = torch.from_numpy(self.mask[b, :n, :n]).bool() if self.mask is not None \
                else torch.ones(n, n).tril().bool()
            for h in range(H):
                q = self.q[b, :n, h * G:(h + 1) * G].double()
                for i in range(n):
                    at = see[i].nonzero().squeeze(1)
                    if at.numel() == 0:
                        continue
                    kk, vv = k[at, h], v[at, h]
                    s = q[i] @ kk.T * self.scale                                   # [G, seen]
                    size = (q[i].abs() @ kk.abs().T * abs(self.scale)).amax(dim=1)  # [G]
                    z = torch.logsumexp(s, dim=1)
                    w = torch.exp(s - z[:, None])
                    o, a = w @ vv, w @ vv.abs()
                    sl = slice(h * G, (h + 1) * G)
                    out[b, i, sl], lse[b, i, sl] = o, z
                    rel = (D + 8) * 2.0 ** -24 * size + 2.0 ** -22 + at.numel() * 2.0 ** -24
                    tol_l[b, i, sl] = rel + 2.0 ** -22 * z.abs()
                    tol_o[b, i, sl] = (2 * rel[:, None] + half + 2.0 ** -22) * a + half * o.abs() + 1e-30
        return out, lse, tol_o, tol_l


def assert_attention(got, want, label=""):
    out, lse, tol_o, tol_l = want
    o, z = got["out"].double().cpu(), got["lse"].double().cpu()
    assert torch.equal(torch.isneginf(z), torch.isneginf(lse)), label
    fin = ~torch.isneginf(lse)
    assert bool(((z - lse).abs()[fin] <= tol_l[fin]).all()), (label, float(((z - lse).abs()[fin] / tol_l[fin]).max()))
    worst = ((o - out).abs() / tol_o.clamp(min=1e-30)).max() if out.numel() else 0.0
    assert bool(((o - out).abs() <= tol_o).all()), (label, float(worst))


def grow(table, refs, seqs, tokens, page_size):
    """cache_resize on numpy arrays, in place; returns the status list."""
    S, M = table.shape
    OK, EDATA, ENOPAGES = 0, 4, 6
    status, grows = [], []
    for s, t in zip(seqs, tokens):
        want = -(-int(t) // page_size)
        if not 0 <= s < S or t < 0 or want > M:
            status.append(EDATA)
            grows.append(None)
            continue
        have = int(np.argmax(np.append(table[s], -1) == -1))
        if any(not 0 <= p < len(refs) for p in table[s, :have]):
            status.append(EDATA)
            grows.append(None)
            continue
        for i in range(want, have):
            refs[table[s, i]] -= 1
            table[s, i] = -1
        status.append(OK)
        grows.append((s, have, want) if want > have else None)
    free = list(np.nonzero(refs == 0)[0])
    asked = 0
    for f, g in enumerate(grows):
        if g is None:
            continue
        s, have, want = g
        asked += want - have
        if asked > len(free):
            status[f] = ENOPAGES
            continue
        for i, p in enumerate(free[asked - (want - have):asked]):
            table[s, have + i] = p
            refs[p] = 1
    return status


def fork(k, v, table, lens, refs, src, dst, page_size):
    """cache_fork on CPU tensors (k, v) and numpy arrays, in place."""
    S, M = table.shape
    OK, EDATA, ENOPAGES = 0, 4, 6
    old_len, old_table = lens.copy(), table.copy()
    free = list(np.nonzero(refs == 0)[0])
    asked, status = 0, []
    for s, d in zip(src, dst):
        if not (0 <= s < S and 0 <= d < S) or s == d or old_table[d, 0] != -1 or \
                not 0 <= old_len[s] <= M * page_size or \
                any(not 0 <= p < len(refs) for p in old_table[s, :-(-old_len[s] // page_size)]):
            status.append(EDATA)
            continue
        L = int(old_len[s])
        full, rest = L // page_size, L % page_size
        asked += rest > 0
        if rest and asked > len(free):
            status.append(ENOPAGES)
            continue
        table[d, :full] = old_table[s, :full]
        for p in old_table[s, :full]:
            refs[p] += 1
        if rest:
            new, old = free[asked - 1], old_table[s, full]
            table[d, full] = new
            refs[new] = 1
            k[:, new, :rest] = k[:, old, :rest]
            v[:, new, :rest] = v[:, old, :rest]
        lens[d] = L
        status.append(OK)
    return status
