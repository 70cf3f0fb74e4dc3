"""The weighing is two launches of which the second is programmatic: calls of several threads on
one stream, and other work between them, add up as they do one after the other."""

import threading

import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from test_gpu_weigh import Weigh

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,lens", [(128, [300, 40]), (64, [2000] * 20)])
def test_threads_add_up_on_one_stream(D, lens):
    a = Weigh(61, lens, 3, 2, 2, D, 16, "bf16").args()
    start = a["weights"].clone()
    calls, threads = 60, 3
    for _ in range(calls * threads):
        sv.cache_weigh(**a)
    want = a["weights"].clone()
    for _ in range(3):
        a["weights"].copy_(start)
        bad, gate = [], threading.Barrier(threads)

        def work():
            gate.wait()
            for _ in range(calls):
                r = sv.cache_weigh(**a)
                if len(bad) < 3 and r["status"].shape[0] != len(lens):
                    bad.append(r)

        ts = [threading.Thread(target=work) for _ in range(threads)]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
        torch.cuda.synchronize()
        assert not bad and torch.equal(a["weights"], want)


def test_work_between_calls():
    """Each call sees what the stream did to the weights, the queries and the lengths before it."""
    w = Weigh(62, [500, 70, 9], 2, 2, 2, 64, 16, "bf16")
    a = w.args()
    start = a["weights"].clone()
    for i in range(50):
        a["weights"].zero_()
        a["q"].mul_(1.0)
        r = sv.cache_weigh(**a)["status"]
        a["weights"].add_(start)
    assert r.tolist() == [0] * 3
    off = (a["weights"].double().cpu() - w.want).abs()
    assert (off <= w.tol + 2.0 ** -23 * w.want).all()
