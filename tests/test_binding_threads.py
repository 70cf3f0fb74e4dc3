"""Threads that call on one stream, on the host alone: the library is replaced by
one that records when calls are inside it. A call takes its workspace and
enqueues its kernels with no other call of the stream in between; calls on other
streams do not wait."""

import threading
import time
import types

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv


class Library:
    """Every entry point takes a moment; .most: calls inside at one time, by stream (their last argument)."""

    def __init__(self, meet=None):
        self.inside, self.most, self.lock, self.meet = {}, {}, threading.Lock(), meet

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 256

        def call(*a):
            stream = getattr(a[-1], "value", a[-1])
            with self.lock:
                self.inside[stream] = self.inside.get(stream, 0) + 1
                self.most[stream] = max(self.most.get(stream, 0), self.inside[stream])
            if self.meet:
                self.meet.wait(5)   # all calls inside at once, or an error
            time.sleep(0.005)
            with self.lock:
                self.inside[stream] -= 1
            return 0
        return call


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


class Staging:
    host, device = False, types.SimpleNamespace(index=-1, type="cpu")   # (get_device() of a host tensor is -1)

    def __init__(self, ref):
        pass

    def dev(self, t, dtype=None):
        return t

    def out(self, shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype)

    def back(self, d):
        return d


CACHE = torch.zeros(1, 4, 16, 1, 8)
I32 = dict(dtype=torch.int32)
Z = torch.zeros(2, 3, 5)
CALLS = {
    "tree_attention": lambda: sv.tree_attention(torch.zeros(2, 1, 1, 8), CACHE[0], CACHE[0], torch.zeros(2, 2, **I32),
                                                torch.zeros(2, **I32)),
    "cache_fork": lambda: sv.cache_fork(CACHE, CACHE, torch.zeros(2, 2, **I32), torch.zeros(2, **I32),
                                        torch.zeros(4, **I32), torch.zeros(1, **I32), torch.ones(1, **I32)),
    "verify": lambda: sv.verify(Z, Z[:, :2], torch.zeros(2, 2, **I32)),
    "verify_lenient": lambda: sv.verify(Z, Z[:, :2], torch.zeros(2, 2, **I32), lenience=0.5),
    "verify_tree": lambda: sv.verify_tree(Z, *[torch.zeros(2, 3, **I32)] * 3, 2),
    "acceptance_rate": lambda: sv.acceptance_rate(Z, Z[:, :2]),
    "verify_mentor": lambda: sv.verify_mentor(Z, Z[:, :2], torch.zeros(2, 2, **I32)),
    "sample": lambda: sv.sample(Z),
}


@pytest.fixture
def on_host(monkeypatch):
    """The binding with host tensors; .raw[thread]: the raw handle of its current stream."""
    raw = threading.local()
    buffers = {}
    monkeypatch.setattr(sv, "_Staging", Staging)
    monkeypatch.setattr(sv, "_given", lambda out, index, want: {})
    monkeypatch.setattr(sv, "_cache_args", lambda k, v, layered: (b"", k.shape, 0))
    monkeypatch.setattr(sv, "_attention_bytes", lambda *a: 256)
    monkeypatch.setattr(sv, "_raw_stream", lambda index: raw.value)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(raw.value))
    monkeypatch.setattr(sv, "workspace", lambda n, dev, stream: buffers.setdefault(stream.cuda_stream, torch.empty(n)))

    def use(lib):
        monkeypatch.setattr(sv, "load_library", lambda path=None: lib)
        monkeypatch.setattr(sv, "_library", lambda: lib)
        return raw
    return use


def _threads(raw, jobs):
    errors = []

    def work(stream, call):
        raw.value = stream
        try:
            call()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
    ts = [threading.Thread(target=work, args=j) for j in jobs]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_one_stream_take_turns(on_host, name):
    lib = Library()
    raw = on_host(lib)
    _threads(raw, [(1234, CALLS[name])] * 4 + [(1234, CALLS["tree_attention"])] * 2)
    assert lib.most == {1234: 1}


def test_calls_on_other_streams_do_not_wait(on_host):
    lib = Library(threading.Barrier(3))
    raw = on_host(lib)
    _threads(raw, [(s, CALLS[n]) for s, n in ((11, "tree_attention"), (12, "cache_fork"), (13, "verify"))])
    assert lib.most == {11: 1, 12: 1, 13: 1}


def test_a_failing_call_gives_its_turn_back(on_host, monkeypatch):
    lib = Library()
    raw = on_host(lib)
    raw.value = 99

    def broken(*a):
        raise RuntimeError("no workspace")
    with monkeypatch.context() as m:
        m.setattr(sv, "workspace", broken)
        for name in ("verify", "tree_attention"):
            with pytest.raises(RuntimeError):
                CALLS[name]()
    _threads(raw, [(99, CALLS["verify"]), (99, CALLS["tree_attention"])])
    assert lib.most == {99: 1}
