"""Rows split over a cluster of blocks, for every number of alternatives: each part leaves as
many to the first block as are asked for, by as many threads of a warp."""

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from test_gpu_logprobs import logits, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,V,B", [("f32", 128256, 3), ("f32", 32000, 200), ("bf16", 128256, 3), ("bf16", 8009, 3)])
def test_every_number_of_alternatives(dtype, V, B):
    """Eight parts, two, eight, four: those of a call with fewer are the first of one with more."""
    z, t = logits(7, B, 2, V, dtype), tokens(7, B, 2, V)
    most = sv.token_logprobs(z, t, top=32)
    order = z.float().sort(stable=True, dim=-1, descending=True).indices[..., :32]
    assert torch.equal(most["top_tokens"].long(), order)
    for top in range(32):
        r = sv.token_logprobs(z, t, top=top)
        for k in ("logprob", "rank", "entropy", "status"):
            assert torch.equal(r[k], most[k]), (k, top)
        if top:
            for k in ("top_tokens", "top_logprobs"):
                assert torch.equal(r[k], most[k][..., :top]), (k, top)
