"""Pages that several sequences hold are not written: a forked sequence that was
shortened to inside a shared page, appending and compacting with the counts."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def ints(*x):
    return torch.tensor(x, **I32)


class Pool:
    """Sequence 0 holds 40 tokens (pages of 16); 1 and 2 are its forks."""

    def __init__(self, dtype=torch.float32, layers=2, pages=20):
        g = torch.Generator(device="cuda").manual_seed(1)
        self.k = torch.randn(layers, pages, 16, 2, 64, generator=g, device="cuda").to(dtype)
        self.v = torch.randn(layers, pages, 16, 2, 64, generator=g, device="cuda").to(dtype)
        self.table, self.refs, self.len = torch.full((5, 6), -1, **I32), torch.zeros(pages, **I32), torch.zeros(5, **I32)
        self.resize([0], [40])
        self.len[0] = 40
        self.fork([0, 0], [1, 2])
        assert self.refs[:5].tolist() == [3, 3, 1, 1, 1]

    def resize(self, seqs, tokens):
        assert not sv.cache_resize(self.table, self.refs, ints(*seqs), ints(*tokens), 16)["status"].any()

    def fork(self, src, dst):
        assert not sv.cache_fork(self.k, self.v, self.table, self.len, self.refs, ints(*src), ints(*dst))["status"].any()

    def append(self, seqs, x, refs=True):
        return sv.cache_append(x, -x, self.k[0], self.v[0], self.table[seqs], self.len[seqs],
                               page_refs=self.refs if refs else None)["status"].tolist()

    def rows(self, s, n):
        at = torch.arange(n, device="cuda")
        return self.k[0, self.table[s, at // 16].long(), at % 16].clone()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_to_a_shared_page_is_refused(dtype):
    p = Pool(dtype)
    p.resize([1], [20])
    p.len[1] = 20
    p.resize([2], [60])
    x = torch.randn(3, 3, 2, 64, device="cuda").to(dtype)
    before = p.rows(0, 40)
    seqs = torch.tensor([1, 2, 0])
    assert p.append(seqs, x) == [4, 0, 0]   # the others' last pages are their own
    assert torch.equal(p.rows(0, 40), before)
    assert torch.equal(p.rows(2, 43)[40:], x[1]) and torch.equal(p.rows(0, 43)[40:], x[2])
    # forked into an empty sequence instead, and released
    p.fork([1], [3])
    p.resize([1, 3], [0, 23])
    mine = p.rows(3, 20)
    assert p.append(torch.tensor([3]), x[:1]) == [0]
    assert torch.equal(p.rows(0, 40), before) and torch.equal(p.rows(3, 23)[20:], x[0])
    assert torch.equal(p.rows(3, 20), mine) and torch.equal(mine, before[:20])
    # shortened to the end of a shared page: the next one is its own
    p.resize([2], [32])
    p.len[2] = 32
    p.resize([2], [35])
    assert p.append(torch.tensor([2]), x[1:2]) == [0]
    assert torch.equal(p.rows(0, 40), before)
    # a page that nobody holds is not written either
    p.refs[p.table[2, 2].long()] = 0
    assert p.append(torch.tensor([2]), x[1:2]) == [4]


def test_compact_into_a_shared_page_is_refused():
    p = Pool()
    p.resize([1], [20])
    p.len[1] = 20
    k, v = p.k.clone(), p.v.clone()

    def compact(seqs, acc, path):
        r = sv.cache_compact(p.k, p.v, p.table[seqs], p.len[seqs], ints(*acc),
                             None if path is None else torch.tensor(path, **I32), page_refs=p.refs)
        return r["status"].tolist(), r["cache_len"].tolist()

    one = torch.tensor([1])
    assert compact(one, [2], [[0, 3, 5]]) == ([4], [-1])
    assert torch.equal(p.k, k) and torch.equal(p.v, v)
    assert compact(one, [2], None) == ([0], [23])               # a chain: nothing is written
    assert compact(one, [2], [[0, 1, 2]]) == ([0], [23])        # in place already
    assert torch.equal(p.k, k) and torch.equal(p.v, v)
    # the root and its child lie in a shared page, in place; what moves goes to a page of its own
    p.len[2] = 30
    p.resize([2], [48])
    assert compact(torch.tensor([2]), [3], [[0, 1, 5, 9]]) == ([0], [34])
    own = p.table[2, 2].item()
    np.testing.assert_array_equal(p.k[:, own, 0].cpu().numpy(), k[:, own, 3].cpu().numpy())
    np.testing.assert_array_equal(p.v[:, own, 1].cpu().numpy(), v[:, own, 7].cpu().numpy())
    shared = p.table[2, 1].item()
    assert torch.equal(p.k[:, shared], k[:, shared])


def test_counts_are_checked():
    p = Pool()
    x = torch.zeros(1, 1, 2, 64, device="cuda")
    for bad in (p.refs.long(), p.refs[:19], p.refs.cpu(), torch.zeros(40, **I32)[::2]):
        with pytest.raises(sv.SpecError):
            sv.cache_append(x, x, p.k[0], p.v[0], p.table[:1], p.len[:1], page_refs=bad)
        with pytest.raises(sv.SpecError):
            sv.cache_compact(p.k, p.v, p.table[:1], p.len[:1], ints(1), page_refs=bad)
