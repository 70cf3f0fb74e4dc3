"""Threads that call on one stream at the same time: the outputs of calls one after the other."""

import threading

import pytest
import torch

import paged
import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu


def test_attention_and_forks_of_several_threads():
    """Split units (their pieces pass through the workspace), head sizes that share a
    kernel, and forks (their copies do), all on the default stream."""
    shapes = [([3000, 40], 5, 2, 4, 128, "bf16"), ([2000], 9, 4, 1, 64, "f32"), ([2500, 7], 6, 4, 1, 32, "f32"),
              ([1500], 30, 2, 4, 128, "f32")]
    cases = [paged.Case(61 + i, lens, N, H, G, D, 16, dt, False).args() for i, (lens, N, H, G, D, dt) in enumerate(shapes)]
    want = [sv.tree_attention(with_lse=True, **a) for a in cases]
    i32 = dict(dtype=torch.int32, device="cuda")
    k0 = torch.randn(4, 40, 16, 2, 64, device="cuda")
    src, dst = torch.zeros(3, **i32), torch.tensor([1, 2, 3], **i32)

    def pool():
        table, refs, lens = torch.full((4, 4), -1, **i32), torch.zeros(40, **i32), torch.zeros(4, **i32)
        table[0, :3] = torch.arange(3, **i32)
        refs[:3] = 1
        lens[0] = 39
        return k0.clone(), -k0, table, lens, refs

    want_pool = pool()
    sv.cache_fork(*want_pool, src, dst)
    torch.cuda.synchronize()
    errors = []

    def attention(i):
        for _ in range(40):
            got = sv.tree_attention(with_lse=True, **cases[i])
            if not all(torch.equal(got[k], want[i][k]) for k in got):
                errors.append(i)

    def forks():
        for _ in range(40):
            p = pool()
            sv.cache_fork(*p, src, dst)
            if not all(torch.equal(a, b) for a, b in zip(p, want_pool)):
                errors.append("fork")

    threads = [threading.Thread(target=attention, args=(i,)) for i in range(4)] + [threading.Thread(target=forks)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
