"""Tree attention repeats itself to the bit whatever ran before it: row tiles
that are partly filled, after calls that leave other queries in shared memory."""

import threading

import pytest
import torch

import paged
import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [("f32", 128), ("f32", 64), ("f32", 192), ("bf16", 96), ("bf16", 128), ("bf16", 64)])
@pytest.mark.parametrize("rows", [5, 17, 61, 125])
def test_absent_rows_have_no_influence(dtype, D, rows):
    def case(n, seed, q_scale):
        return paged.Case(seed, [900] * 10, n, 8, 1, D, 64, dtype, False, q_scale=q_scale).args()

    a = case(rows, 1, 1.5)
    first = sv.tree_attention(with_lse=True, **a)
    for q_scale in (1e-3, 30.0, 1e3, 1e6):
        full = case(-(-rows // 64) * 64, 2, q_scale)
        full["q"] = full["q"].abs()
        sv.tree_attention(**full)
        again = sv.tree_attention(with_lse=True, **a)
        for k in ("out", "lse"):
            assert torch.equal(again[k], first[k]), (k, q_scale)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_a_thread_s_first_call(dtype, D):
    """The same bits as in the main thread, and so the same kernel."""
    a = paged.Case(3, [3000, 40], 5, 2, 4, D, 16, dtype, False).args()
    want = sv.tree_attention(with_lse=True, **a)
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        t = threading.Thread(target=lambda: got.append(sv.tree_attention(with_lse=True, **a)))
        t.start()
        t.join()
    assert len(got) == 3
    for r in got:
        for k in ("out", "lse", "status"):
            assert torch.equal(r[k], want[k]), k
