"""Every source with kernels checks indices in the debug build and has its failures read."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_verification_05_gb300", "csrc")
KERNELS = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and "__global__" in open(os.path.join(CSRC, f)).read())


@pytest.mark.parametrize("name", [f for f in KERNELS if f != "api.cu"])
def test_source_is_checked_and_read(name):
    """(api.cu's kernel writes one word a thread below its bound.)"""
    text = open(os.path.join(CSRC, name)).read()
    assert re.search(r"\bSV_IN(_SEQ)?\(", text)
    readers = re.findall(r"SV_DEBUG_READER\((\w+)\)", text)
    assert len(readers) == 1
    assert f"debug_read_{readers[0]}" in open(os.path.join(CSRC, "api.cu")).read()
