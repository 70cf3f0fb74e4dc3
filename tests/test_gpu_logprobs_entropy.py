"""Entropies and alternatives of token_logprobs, closely, at ordinary and extreme temperatures.

With y = (z - m) / T and p = e^y / S: H = ln S - sum p y. A term's weight is off by the
exponential's 2^-22 and by 2^-24 |t| of its exponent t in octaves (what counts has |t| < 30:
2^-19.6 with ln 2), a sum's by A 2^-24 for the A additions on a term's way (16 of a thread's
batch, one a batch, under 20 of the trees: at most 40 for rows to 8000, 100 for rows to
262144). Together e = 2^-18 and 2^-16.8. H is a sum of ln S (off by e) and of a quotient of
sums (off by 2 e of itself), which lies in 0 .. ln V: (1 + 2 ln V) e, and 2^-22 of H for the
last roundings. A log probability is off by e and by four roundings of itself, 2^-22."""

import math

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from test_gpu_logprobs import logits, tokens

pytestmark = pytest.mark.gpu


def check(z, t, top, T):
    V = z.shape[-1]
    e = 2.0 ** -18 if V <= 8000 else 2.0 ** -16.8
    r = sv.token_logprobs(z, t, top=top, temperature=T)
    y = z.double()
    y = (y - y.amax(-1, keepdim=True)) / T
    lp = y - torch.logsumexp(y, -1, keepdim=True)
    p = lp.exp()
    H = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    off = (r["entropy"].double() - H).abs()
    assert (off <= (1 + 2 * math.log(V)) * e + 2.0 ** -22 * H).all(), float(off.max())
    order = z.float().sort(stable=True, dim=-1, descending=True).indices[..., :top]
    assert torch.equal(r["top_tokens"].long(), order)
    for got, want in ((r["top_logprobs"], lp.gather(-1, order)), (r["logprob"], lp.gather(-1, t.long()[..., None])[..., 0])):
        low = want < -3.4e38   # (float32 has no room)
        assert torch.isneginf(got[low]).all()
        assert ((got.double() - want).abs()[~low] <= e + 2.0 ** -22 * want.abs()[~low]).all()
    assert r["status"].tolist() == [0] * z.shape[0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1e-30, 1e-5, 1e-3, 0.05, 0.7, 1.0, 3.0, 1e4, 1e30])
def test_temperatures(dtype, T):
    z, t = logits(41, 3, 2, 3001, dtype), tokens(41, 3, 2, 3001)
    z[1, 0, 7:11] = z[1, 0].amax()   # several likeliest ones: ln of their number at the lowest temperatures
    z[2, 1] = z[2, 1].round()
    t[0, 0] = z[0, 0].argmax()
    check(z, t, 6, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V", [(2, 32000), (400, 32016), (2, 128256), (2, 262144)])
@pytest.mark.parametrize("T", [0.01, 1.0, 100.0])
def test_long_rows(dtype, B, V, T):
    check(logits(42, B, 2, V, dtype), tokens(42, B, 2, V), 5, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_logits(dtype):
    """Maxima far from zero: the exponents' reference is rounded, or not taken from a product at all."""
    for add in (-3e4, 1e3, 2e5, 1e6, 3e7):
        z, t = logits(43, 2, 2, 5003, dtype, sd=max(2.5, abs(add) * 2.0 ** -12)), tokens(43, 2, 2, 5003)
        check((z.float() + add).to(z.dtype), t, 4, 1.0)


def test_equal_logits():
    for V in (2, 1000, 32000):
        z, t = torch.full((1, 3, V), -3.25, device="cuda"), tokens(44, 1, 3, V)
        check(z, t, 2, 0.3)
