"""The cache's operators together, as examples/paged_tree_decode.py runs them:
draft trees over a forked, paged cache give the tokens of plain decoding."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_tree_decode.py")
    spec = importlib.util.spec_from_file_location("paged_tree_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("branches,prompt_tokens,wrong", [(3, 37, 0.25), (1, 1, 0.0), (5, 48, 0.6)])
def test_trees_give_the_tokens_of_plain_decoding(example, branches, prompt_tokens, wrong):
    want, got, calls = example.run(branches=branches, steps=24, prompt_tokens=prompt_tokens, wrong=wrong)
    assert (want == got).all()
    assert calls < 24 if wrong < 0.5 else calls <= 24
