"""The Python binding's host side, without a GPU: which device a call runs on."""

import contextlib

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv


class Used(Exception):
    """A tensor was looked at; .current: the device that was current then."""


class OnDevice1:
    """A stand-in for a tensor on cuda:1 that raises at its first real use."""

    is_cuda = True
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1

    def __getattr__(self, name):
        e = Used(name)
        e.current = CURRENT[0]
        raise e


CURRENT = [0]


@pytest.fixture
def two_devices(monkeypatch):
    @contextlib.contextmanager
    def device(d):
        before, CURRENT[0] = CURRENT[0], torch.device("cuda", d).index if isinstance(d, int) else d.index
        try:
            yield
        finally:
            CURRENT[0] = before

    monkeypatch.setattr(sv, "_device", lambda: CURRENT[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(sv, "load_library", lambda path=None: object())
    monkeypatch.setattr(sv, "_library", lambda: object())


T = OnDevice1()
CALLS = {
    "verify": lambda: sv.verify(T, T, T),
    "verify by name": lambda: sv.verify(draft_tokens=T, draft=T, target=T),
    "verify_tree": lambda: sv.verify_tree(T, T, T, T, 3),
    "tree_build": lambda: sv.tree_build(T, T, 10, 4),
    "acceptance_rate": lambda: sv.acceptance_rate(T, T),
    "verify_mentor": lambda: sv.verify_mentor(T, T, T),
    "sample": lambda: sv.sample(T),
    "tree_attention": lambda: sv.tree_attention(torch.zeros(1, 1, 1, 8), T, T, T, T),
    "tree_attention by name": lambda: sv.tree_attention(torch.zeros(1, 1, 1, 8), v_cache=T, k_cache=T, page_table=T,
                                                        cache_len=T),
    "cache_append": lambda: sv.cache_append(T, T, T, T, T, T),
    "cache_compact": lambda: sv.cache_compact(T, T, T, T, T),
    "cache_resize": lambda: sv.cache_resize(T, T, None, T, 16),
    "cache_fork": lambda: sv.cache_fork(T, T, T, T, T, T, T),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_run_on_their_tensors_device(two_devices, name):
    CURRENT[0] = 0
    with pytest.raises(Used) as e:
        CALLS[name]()
    assert e.value.current == 1
    assert CURRENT[0] == 0
    CURRENT[0] = 1
    with pytest.raises(Used) as e:
        CALLS[name]()
    assert e.value.current == 1 and CURRENT[0] == 1
    CURRENT[0] = 0


@pytest.mark.parametrize("name", ["verify", "tree_attention", "cache_resize"])
def test_what_is_no_tensor_raises_as_before(two_devices, name):
    fn = getattr(sv, name)
    with pytest.raises((TypeError, AttributeError)):
        fn()
    with pytest.raises((TypeError, AttributeError)):
        fn(*[None] * 5)


def test_signatures_and_names_are_kept():
    import inspect

    assert list(inspect.signature(sv.tree_attention).parameters)[:3] == ["q", "k_cache", "v_cache"]
    assert sv.cache_fork.__name__ == "cache_fork" and sv.cache_fork.__doc__


def test_given_outputs_are_checked():
    i32, f32 = torch.int32, torch.float32
    want = dict(out=((2, 3, 4, 8), torch.bfloat16), lse=((2, 3, 4), f32), status=((2,), i32))
    good = dict(out=torch.zeros(2, 3, 4, 8, dtype=torch.bfloat16), lse=torch.zeros(2, 3, 4), status=torch.zeros(2, dtype=i32))
    host = -1   # get_device() of a host tensor: the checks are the same
    assert sv._given(None, host, want) == {}
    o = sv._given(good, host, want)
    assert o == good and o is not good
    assert sv._given({"status": good["status"]}, host, want) == {"status": good["status"]}
    for key, bad in (("out", good["out"][:1]), ("out", good["out"].float()), ("out", good["out"].flatten()),
                     ("out", good["out"].transpose(1, 2).contiguous().transpose(1, 2)), ("lse", good["lse"].double()),
                     ("lse", torch.zeros(2, 3, 8)[..., ::2]), ("lse", torch.zeros(2, 4, 3)), ("status", torch.zeros(2)),
                     ("status", torch.zeros(2, dtype=torch.int64)), ("status", torch.zeros(3, dtype=i32))):
        with pytest.raises(sv.SpecError):
            sv._given({**good, key: bad}, host, want)
    with pytest.raises(sv.SpecError):
        sv._given(good, 0, want)   # on the host, for a call on a device
