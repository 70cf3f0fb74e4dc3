"""The bounded cache and the log probabilities at the ends of their ranges: offsets
past 32 bits, the largest pages and groups, extreme temperatures, many rows, calls on
two streams at once. What a call returns there is compared with the same call on small
tensors (equal bits) or with the definition."""

import math

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from test_gpu_evict import Cache
from test_gpu_logprobs import check, logits, tokens
from test_gpu_weigh import Weigh, paths

pytestmark = pytest.mark.gpu


def step(kc, vc, table, q, k, v, dtype):
    """Append, attention, weights and eviction of two sequences over the pages of `table`."""
    lens = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    r = sv.cache_append_rotary(q, k, v, kc[0], vc[0], table, lens, sv.rotary(128))
    o = sv.tree_attention(r["q"], kc[0], vc[0], table, lens, with_lse=True)
    w = torch.zeros(2, kc.shape[3], table.shape[1] * 16, device="cuda")
    s = sv.cache_weigh(r["q"], o["lse"], kc[0], table, lens, w)
    n = k.shape[1]
    e = sv.cache_evict(kc, vc, table, lens + n, w[None], 70, sink=3, recent=20)
    for x in (r, o, s, e):
        assert x["status"].tolist() == [0, 0]
    rows = [kc[0][table[:, :5].long()], vc[0][table[:, :5].long()]]
    return [r["q"], o["out"], o["lse"], w, e["cache_len"], *rows]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pages_past_32_bits(dtype):
    """A pool of more than 2^31 elements, pages at its end."""
    pages, H, D = 140000, 8, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(2, 100, h, D, generator=g, device="cuda").to(dtype) for h in (16, H, H))
    got = []
    for P in (20, pages):
        kc, vc = (torch.empty(1, P, 16, H, D, dtype=dtype, device="cuda") for _ in range(2))
        assert P == 20 or kc.numel() > 2 ** 31
        table = torch.stack([torch.arange(P - 1, P - 8, -1), torch.arange(P - 20, P - 13)]).int().cuda()
        got.append([x.clone() for x in step(kc, vc, table, q, k, v, dtype)])
        del kc, vc
    for a, b in zip(*got):
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


def test_logits_past_32_bits():
    B, P, V = 60, 300, 128256
    z = torch.empty(B, P, V, dtype=torch.bfloat16, device="cuda")
    assert z.numel() > 2 ** 31
    t = torch.full((B, P), -1, dtype=torch.int32, device="cuda")
    z[-1, -3:] = logits(2, 1, 3, V, "bf16")[0]
    t[-1, -3:] = tokens(2, 1, 3, V)[0]
    r = sv.token_logprobs(z, t, top=8)
    one = check(z[-1:, -3:].contiguous(), t[-1:, -3:].contiguous(), 8)
    for x in ("rank", "top_tokens"):
        assert torch.equal(r[x][-1:, -3:], one[x])
    assert (r["logprob"][-1:, -3:] - one["logprob"]).abs().max() < 2.0 ** -15
    assert r["status"].tolist() == [0] * B and (r["logprob"][:-1] == 0).all()


def test_many_rows_of_few_tokens():
    check(logits(3, 1, 20000, 5, "f32"), tokens(3, 1, 20000, 5), 5)
    check(logits(4, 3000, 1, 37, "bf16"), tokens(4, 3000, 1, 37), 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1e-30, 1e-3, 1e4, 1e30])
def test_extreme_temperatures(dtype, T):
    """Nearly one token, nearly all alike: finite or -inf, in order, and adding up."""
    z, t = logits(5, 2, 2, 3001, dtype), tokens(5, 2, 2, 3001)
    t[0, 0] = z[0, 0].argmax()
    r = sv.token_logprobs(z, t, top=4, temperature=T)
    y = (z.double() - z.double().amax(-1, keepdim=True)) / T
    want = (y - torch.logsumexp(y, -1, keepdim=True)).gather(-1, t.long()[..., None])[..., 0]
    got = r["logprob"].double()
    low = want < -3e38   # (float32 has no room)
    assert torch.isneginf(got[low]).all() and r["status"].tolist() == [0, 0]
    # (a difference of two logits times 1 / T: three roundings)
    assert ((got - want).abs()[~low] <= 2.0 ** -15 + 2.0 ** -21 * want.abs()[~low]).all()
    assert (r["entropy"] >= 0).all() and (r["entropy"] <= math.log(3001) + 2.0 ** -10).all()
    assert (r["top_logprobs"][..., 1:] <= r["top_logprobs"][..., :-1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_pages_and_groups(dtype):
    Weigh(21, [700, 255, 0], 3, 1, 2, 128, 256, dtype).check()
    Weigh(22, [40], 5, 1, 128, 64, 256, dtype).check()
    Weigh(23, [300, 20], 2, 1, 100, 128, 8, dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_paths_of_large_groups(dtype):
    import numpy as np

    rng = np.random.default_rng(24)
    accept = np.array([255, 100, 3])
    Weigh(24, [500, 64, 129], 300, 1, 5, 64, 16, dtype, accept, paths(rng, 3, 300, 256, accept)).check()


def test_two_streams_at_once():
    """Calls that share nothing but the library, on two streams."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [[Cache(30 + i + 10 * r, [900, 400, 700], 4, 4, 64, 16) for i in range(2)] for r in range(4)]
    want = [[c.expected([300] * 3, 2, 50) for c in pair] for pair in caches]
    weigh = [Weigh(40 + i, [600, 50], 5, 2, 4, 128, 16, "bf16") for i in range(2)]
    args = [w.args() for w in weigh]
    z, t = logits(50, 8, 4, 32000, "bf16"), tokens(50, 8, 4, 32000)
    alone = sv.token_logprobs(z, t, top=10)
    torch.cuda.synchronize()
    lp = []
    for pair in caches:
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                c = pair[i]
                c.out = sv.cache_evict(c.k, c.v, c.table, c.len, c.w, torch.full((3,), 300, dtype=torch.int32, device="cuda"), 2, 50)
                lp.append(sv.token_logprobs(z, t, top=10))
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            sv.cache_weigh(**args[i])
    torch.cuda.synchronize()
    for pair, w in zip(caches, want):
        for c, (k, v, ww, new) in zip(pair, w):
            assert torch.equal(c.k.cpu(), k) and torch.equal(c.v.cpu(), v) and torch.equal(c.w.cpu(), ww)
            assert c.out["cache_len"].tolist() == new
    for w, a in zip(weigh, args):
        assert ((a["weights"].double().cpu() - w.want).abs() <= w.tol).all()
    for r in lp:
        for x in alone:
            assert torch.equal(r[x], alone[x])
