"""token_logprobs on rows that hold NaN, whatever its bits: a model that breaks down gives
whole rows of them, and the arithmetic of the device gives 0x7FFFFFFF, whose ordered key is
the largest that there is. Such a row's outputs are NaN and -1, its sequence SPEC_EDATA, and
every other row's outputs are the bits that they are without it."""

import math

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from test_gpu_logprobs import logits, tokens

pytestmark = pytest.mark.gpu
BITS = {"f32": (0x7FFFFFFF, 0x7FC00000, 0xFFFFFFFF, 0xFFC00000, 0x7F800001), "bf16": (0x7FFF, 0x7FC0, 0xFFFF, 0x7F81)}


def nan_of(dtype, bits):
    if dtype == "f32":
        return torch.tensor([bits - 2 ** 32 * (bits >> 31)], dtype=torch.int32, device="cuda").view(torch.float32)
    return torch.tensor([bits - 2 ** 16 * (bits >> 15)], dtype=torch.int16, device="cuda").view(torch.bfloat16)


def check(z, clean, t, bad, top):
    """bad: rows (b, p) of z that hold NaN; the others are clean's."""
    want = sv.token_logprobs(clean, t, top=top)
    r = sv.token_logprobs(z, t, top=top)
    at = torch.zeros(t.shape, dtype=torch.bool, device="cuda")
    for b, p in bad:
        at[b, p] = True
    assert (r["status"] == torch.where(at.any(1), sv.SPEC_EDATA, sv.SPEC_OK)).all()
    for k, none in (("logprob", math.nan), ("entropy", math.nan), ("rank", -1), ("top_logprobs", math.nan), ("top_tokens", -1)):
        if k in r:
            x = r[k][at]
            assert (torch.isnan(x) if none != -1 else x == -1).all(), k
            assert torch.equal(r[k][~at], want[k][~at]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,B", [(50, 3), (1500, 3), (32000, 3), (32003, 400), (128256, 2)])
@pytest.mark.parametrize("top", [0, 4, 32])
def test_rows_of_nan(dtype, V, B, top):
    """400 sequences of two rows are a block a row, the few of the long rows eight blocks each."""
    z, t = logits(V, B, 2, V, dtype), tokens(V, B, 2, V)
    for bits in BITS[dtype]:
        x = z.clone()
        x[1, 0] = nan_of(dtype, bits)
        x[B - 1, 1] = nan_of(dtype, bits)
        check(x, z, t, [(1, 0), (B - 1, 1)], top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top", [4, 32])
def test_nan_among_logits(dtype, top):
    """1500 and more of them at a row's start, at its end, in one of its eight parts, at every other
    place, beside nothing but -inf, and two kinds at once."""
    V = 128256
    z, t = logits(2, 7, 1, V, dtype), tokens(2, 7, 1, V)
    for bits in BITS[dtype]:
        x, nan = z.clone(), nan_of(dtype, bits)
        x[0, 0, :1500] = nan
        x[1, 0, -20000:] = nan
        x[2, 0, V // 8:V // 4] = nan
        x[3, 0, 1::2] = nan
        x[4, 0] = -math.inf
        x[4, 0, 1000:4000] = nan
        x[5, 0, ::2] = nan
        x[5, 0, 1::2] = nan_of(dtype, BITS[dtype][0])
        check(x, z, t, [(b, 0) for b in range(6)], top)


@pytest.mark.parametrize("top", [1, 32])
def test_nan_of_the_device(top):
    """The NaN that the device's own arithmetic gives: a product of 0 and infinity."""
    z, t = logits(3, 4, 2, 50257, "f32"), tokens(3, 4, 2, 50257)
    x = z.clone()
    x[2] *= 0.0
    x[2] *= math.inf
    assert torch.isnan(x[2]).all()
    check(x, z, t, [(2, 0), (2, 1)], top)
