"""Which workspace a call gets, on the host alone."""

import contextlib
import types

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv

STREAM = types.SimpleNamespace(cuda_stream=4321)
HOST = torch.device("cpu", 0)


@pytest.fixture
def capturing(monkeypatch):
    state = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state[0])
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: STREAM)
    monkeypatch.setattr(sv, "_ws_cache", {})
    return state


@pytest.mark.parametrize("take", [lambda n: sv.workspace(n, HOST, STREAM), lambda n: sv._scratch(n, HOST, 0, 4321)])
def test_captured_calls_have_buffers_of_their_own(capturing, take):
    a = take(1000)
    assert take(500) is a and take(1000) is a
    capturing[0] = True
    b, c = take(500), take(500)
    assert b is not a and c is not a and b is not c and b.numel() >= 500
    big = take(5000)
    assert big.numel() >= 5000
    capturing[0] = False
    assert take(1000) is a   # nothing of the graph's is left in eager calls
    assert take(5000) is not big
