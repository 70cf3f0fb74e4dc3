"""The device that the bounded cache's calls and token_logprobs run on, without a GPU."""

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from test_binding import CURRENT, T, Used, two_devices  # noqa: F401 (a fixture)

X = torch.zeros(1, 1, 1, 8)
CALLS = {
    "token_logprobs": lambda: sv.token_logprobs(T, T),
    "token_logprobs by name": lambda: sv.token_logprobs(tokens=T, logits=T),
    "cache_append_rotary": lambda: sv.cache_append_rotary(X, T, T, T, T, T, T, T),
    "cache_weigh": lambda: sv.cache_weigh(X, T, T, T, T, T),
    "cache_evict": lambda: sv.cache_evict(T, T, T, T, T, 4),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_run_on_their_tensors_device(two_devices, name):  # noqa: F811
    for current in (0, 1):
        CURRENT[0] = current
        with pytest.raises(Used) as e:
            CALLS[name]()
        assert e.value.current == 1 and CURRENT[0] == current
    CURRENT[0] = 0


@pytest.mark.parametrize("name", ["token_logprobs", "cache_append_rotary", "cache_weigh", "cache_evict"])
def test_names_and_documentation(name):
    fn = getattr(sv, name)
    assert fn.__name__ == name and fn.__doc__ and name in sv.__all__
