"""Captured calls keep their workspaces: replays after the stream's own buffer was
replaced, and beside calls on the stream that was captured."""

import pytest
import torch

import paged
import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu


def test_replays_after_the_workspace_has_grown():
    small = paged.Case(71, [3000], 3, 2, 4, 64, 16, "f32", False).args()     # the smaller workspace of the two
    large = paged.Case(72, [3000], 30, 2, 4, 128, 16, "bf16", False).args()
    i32 = dict(dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = sv.tree_attention(with_lse=True, **small)
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            got = sv.tree_attention(with_lse=True, **small)
        n = sv._ws_cache[(0, stream.cuda_stream)].numel()
        other = sv.tree_attention(with_lse=True, **large)
        assert sv._ws_cache[(0, stream.cuda_stream)].numel() > n
        # what the first buffer was is the next tensors' memory now
        held = [torch.full((n // 4,), 7, **i32) for _ in range(3)]
        g.replay()
        stream.synchronize()
        assert all((t == 7).all() for t in held)
        for k in ("out", "lse", "status"):
            assert torch.equal(got[k], want[k]), k
        # replays on another stream beside calls on the captured one
        beside = torch.cuda.Stream()
        for _ in range(20):
            with torch.cuda.stream(beside):
                g.replay()
            again = sv.tree_attention(with_lse=True, **large)
            torch.cuda.synchronize()
            for k in ("out", "lse", "status"):
                assert torch.equal(got[k], want[k]) and torch.equal(again[k], other[k]), k
