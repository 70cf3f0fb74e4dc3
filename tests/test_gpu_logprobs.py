"""token_logprobs against the definition in 64 bits.

Tolerances. A log probability is (z - m) / T - ln S: three roundings of y = (z -
m) / T, 2^-24 |y| each, and S, whose terms are off by 2^-22 (the exponential, 2
units) and 2^-24 |t| of their exponent t, and which a thread sums by batches of 16
before it adds the batches (64 of them at the most), threads and parts in trees of
under 20 additions: far fewer than 276 roundings of 2^-24 on any way, below 2^-15 if
all went the same way. Entropies add sum w t / S, off by that share of itself, at most
ln V + |ln S| each.
"""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def reference(z, tokens, top, T):
    """z [B, P, V] float64 of finite values and -inf; good rows only."""
    B, P, V = z.shape
    o = {k: np.zeros((B, P)) for k in ("logprob", "entropy")}
    o["rank"] = np.full((B, P), -1)
    o["top_tokens"], o["top_logprobs"] = np.full((B, P, top), -1), np.full((B, P, top), -np.inf)
    for b in range(B):
        for p in range(P):
            x = tokens[b, p]
            if x < 0:
                continue
            y = (z[b, p] - z[b, p].max()) / T
            w = np.exp(y)
            lp = y - math.log(w.sum())
            o["logprob"][b, p] = lp[x]
            o["entropy"][b, p] = -(w[w > 0] / w.sum() * lp[w > 0]).sum()
            o["rank"][b, p] = (z[b, p] > z[b, p, x]).sum() + (z[b, p, :x] == z[b, p, x]).sum()
            order = np.lexsort((np.arange(V), -z[b, p]))[:top]
            o["top_tokens"][b, p], o["top_logprobs"][b, p] = order, lp[order]
    return o


def close(got, want, slack=2.0 ** -15, rel=2.0 ** -21):
    got = got.double().cpu().numpy()
    assert (np.isneginf(got) == np.isneginf(want)).all()
    f = np.isfinite(want)
    off = np.abs(got[f] - want[f])
    assert (off <= slack + rel * np.abs(want[f])).all(), off.max()


def check(z, tokens, top, T=1.0):
    r = sv.token_logprobs(z, tokens, top=top, temperature=T)
    want = reference(z.double().cpu().numpy(), tokens.cpu().numpy(), top, T)
    assert r["status"].cpu().tolist() == [0] * z.shape[0]
    assert (r["rank"].cpu().numpy() == want["rank"]).all()
    close(r["logprob"], want["logprob"])
    close(r["entropy"], want["entropy"], slack=2.0 ** -15 * (2 + 2 * math.log(z.shape[-1])))
    if top:
        assert (r["top_tokens"].cpu().numpy() == want["top_tokens"]).all()
        close(r["top_logprobs"], want["top_logprobs"])
    else:
        assert "top_tokens" not in r
    return r


def logits(seed, B, P, V, dtype, sd=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (sd * torch.randn(B, P, V, generator=g, device="cuda")).to(DT[dtype])


def tokens(seed, B, P, V):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, V, (B, P), generator=g, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,P,V,top,T", [
    (1, 1, 1, 1, 1.0), (2, 1, 2, 2, 0.5), (1, 3, 7, 5, 2.0), (3, 2, 31, 31, 1.0), (2, 5, 100, 32, 1.3), (1, 5, 1000, 0, 1.0),
    (2, 3, 4099, 20, 0.7), (1, 5, 32000, 5, 1.0), (70, 3, 32001, 8, 1.0), (2, 2, 65537, 32, 1.0), (3, 2, 128256, 20, 1.0),
    (1, 2, 262144, 32, 0.9), (1, 1, 262143, 1, 1.0), (400, 2, 513, 3, 1.0)])
def test_against_the_definition(dtype, B, P, V, top, T):
    check(logits(V + B, B, P, V, dtype), tokens(V, B, P, V), top, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [33, 1000, 32016, 70001])
def test_ties_and_orders(dtype, V):
    """Few distinct values, equal logits, sorted rows, the same value with both signs of zero."""
    z = torch.stack([torch.round(logits(1, 1, V, 1, dtype).view(V).float()),
                     torch.zeros(V, device="cuda"),
                     torch.linspace(-4, 4, V, device="cuda"), torch.linspace(4, -4, V, device="cuda"),
                     torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0),
                     torch.where(torch.arange(V, device="cuda") < V - 3, 1.0, 2.0)])[None].to(DT[dtype])
    for at in (0, V // 2, V - 1):
        check(z, torch.full((1, z.shape[1]), at, dtype=torch.int32, device="cuda"), 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [65, 32000, 128256])
def test_masked_logits(dtype, V):
    """-inf and the type's lowest value: most of a row, all but one, and what the token itself is."""
    z = logits(3, 1, 6, V, dtype)
    low = torch.finfo(DT[dtype]).min
    z[0, 0, V // 3:] = -math.inf
    z[0, 1, 1:] = -math.inf
    z[0, 2, :-1] = -math.inf
    z[0, 3, 10:] = low
    z[0, 4] = low
    z[0, 5, ::2] = -math.inf
    for at in (0, 12, V - 1):
        t = torch.full((1, 6), at, dtype=torch.int32, device="cuda")
        r = sv.token_logprobs(z, t, top=20)
        zz = z.double().cpu().numpy()
        want = reference(zz, t.cpu().numpy(), 20, 1.0)
        for k in ("rank", "top_tokens"):
            assert (r[k].cpu().numpy() == want[k]).all(), k
        for k in ("logprob", "top_logprobs"):
            close(r[k], want[k])
        close(r["entropy"], want["entropy"], slack=2.0 ** -10)
        assert r["status"].tolist() == [0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [50, 32016, 128256])
def test_bad_rows_and_tokens(dtype, V):
    z, t = logits(4, 6, 3, V, dtype), tokens(5, 6, 3, V)
    z[0, 1, V // 2] = math.nan
    z[1, 0, 0] = math.inf
    z[2, 2] = -math.inf
    z[3, 1] = math.nan
    t[4, 0] = V
    t[5, 1] = -2
    bad = [(0, 1), (1, 0), (2, 2), (3, 1), (4, 0), (5, 1)]
    r = sv.token_logprobs(z, t, top=4)
    assert r["status"].tolist() == [sv.SPEC_EDATA] * 6
    for b in range(6):
        for p in range(3):
            if (b, p) in bad:
                assert torch.isnan(r["logprob"][b, p]) and torch.isnan(r["entropy"][b, p]) and r["rank"][b, p] == -1
                assert torch.isnan(r["top_logprobs"][b, p]).all() and (r["top_tokens"][b, p] == -1).all()
            else:
                want = reference(z[b:b + 1, p:p + 1].double().cpu().numpy(), t[b:b + 1, p:p + 1].cpu().numpy(), 4, 1.0)
                assert (r["top_tokens"][b, p].cpu().numpy() == want["top_tokens"][0, 0]).all()
                close(r["logprob"][b:b + 1, p:p + 1], want["logprob"])
    one = sv.token_logprobs(z[:, 1:2].contiguous(), t[:, 1:2].contiguous())   # a row a sequence
    assert one["status"].tolist() == [sv.SPEC_EDATA, 0, 0, sv.SPEC_EDATA, 0, sv.SPEC_EDATA]


def test_rows_without_a_token_are_not_read():
    z, t = logits(6, 4, 5, 32000, "bf16"), tokens(7, 4, 5, 32000)
    for b in range(4):
        t[b, b + 1:] = -1
        z[b, b + 1:] = math.nan
    r = check(z.nan_to_num(0.0), t, 6)
    again = sv.token_logprobs(z, t, top=6)
    for k in r:
        assert torch.equal(r[k], again[k]), k
    none = sv.token_logprobs(z, torch.full_like(t, -1), top=2)
    assert (none["logprob"] == 0).all() and (none["top_tokens"] == -1).all() and none["status"].tolist() == [0] * 4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_start_anywhere(dtype):
    """Logits aligned to their element only, vocabularies of any size: every offset of a row in 16 bytes."""
    for V in (999, 4097, 33003):
        for off in range(1, 8):
            flat = logits(off, 1, 1, 3 * V + off, dtype).view(-1)
            z = flat[off:].view(1, 3, V)
            assert z.data_ptr() % 16 != 0 or off * z.element_size() % 16 == 0
            check(z, tokens(off, 1, 3, V), 7)


def test_results_repeat_and_do_not_depend_on_the_batch():
    z, t = logits(8, 64, 8, 32000, "f32"), tokens(9, 64, 8, 32000)
    a, b = sv.token_logprobs(z, t, top=20), sv.token_logprobs(z, t, top=20)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    one = sv.token_logprobs(z[5:6], t[5:6], top=20)
    for k in ("rank", "top_tokens"):
        assert torch.equal(a[k][5], one[k][0])
    assert (a["logprob"][5] - one["logprob"][0]).abs().max() < 2.0 ** -15


def test_streams_graphs_and_host_tensors():
    z, t = logits(10, 3, 4, 5003, "bf16"), tokens(11, 3, 4, 5003)
    want = sv.token_logprobs(z, t, top=5)
    host = sv.token_logprobs(z.cpu(), t.cpu(), top=5)
    for k in want:
        assert not host[k].is_cuda and torch.equal(want[k].cpu(), host[k]), k
    assert torch.equal(sv.token_logprobs(z, t.long(), top=5)["logprob"], want["logprob"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = sv.token_logprobs(z, t, top=5)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sv.token_logprobs(z, t, top=5)
    z2 = logits(12, 3, 4, 5003, "bf16")
    want2 = sv.token_logprobs(z2, t, top=5)
    z.copy_(z2)
    g.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(other[k], want[k]) and torch.equal(out[k], want2[k]), k


def test_with_a_verification_step():
    """verify's tokens with its target: the emitted tokens' rows, nothing after them."""
    zt, zd = logits(13, 5, 4, 1000, "f32"), logits(14, 5, 3, 1000, "f32")
    d = sv.sample(zd, seed=3)["tokens"]
    r = sv.verify(zt, zd, d, seed=4)
    lp = check(zt, r["tokens"], 3)
    n = r["accepted"] + 1
    assert ((lp["rank"] >= 0).sum(1) == n).all()


def test_debug_build_agrees():
    z, t = logits(15, 3, 2, 2049, "f32"), tokens(16, 3, 2, 2049)
    a = sv.token_logprobs(z, t, top=9)
    with sv.use_library(sv.DEBUG_LIB_PATH):
        b = sv.token_logprobs(z, t, top=9)
        assert sv.load_library().spec_debug_failures(None) == 0
    for k in a:
        assert torch.equal(a[k], b[k]), k
