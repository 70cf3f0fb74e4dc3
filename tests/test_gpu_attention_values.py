"""Tree attention and the values of its inputs: infinities in the committed
context, values near the type's largest, and how exact the outputs are."""

import math

import pytest
import torch

import paged
import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu


def _put(c, b, t, head, col, x):
    c.v[c.table[b, t // c.ps], t % c.ps, head, col] = x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_scale", [0.0, 0.1, 1.5, 5.0])
@pytest.mark.parametrize("D,N,G", [(64, 20, 4), (128, 20, 4), (128, 40, 8), (128, 1, 2)])
def test_infinite_values_of_the_context(D, N, G, q_scale, dtype):
    """An infinity in one element of a context position's values: that output
    column of every row, whatever the row's weights (equal ones, flat and peaked
    rows; no weight underflows: scores lie less than 90 apart); elsewhere the
    outputs are those without it."""
    c = paged.Case(31, [300, 130, 700], N, 2, G, D, 16, dtype, True, q_scale=q_scale)
    want = c.expected()
    spots = [(0, 3, 0, 3, math.inf), (0, 77, 1, 60, -math.inf), (0, 299, 0, 17, -math.inf), (1, 0, 0, 5, math.inf),
             (1, 129, 1, 9, math.inf), (2, 128, 0, 33, math.inf), (2, 511, 1, 1, -math.inf), (2, 640, 0, 2, math.inf)]
    for b, t, h, col, x in spots:
        _put(c, b, t, h, col, x)
    out = sv.tree_attention(**c.args())["out"].double().cpu()
    for b, t, h, col, x in spots:
        rows = slice(h * G, (h + 1) * G)
        assert (out[b, :, rows, col] == x).all(), (b, t, h, col, x)
        out[b, :, rows, col] = want[0][b, :, rows, col] = 0
    assert ((out - want[0]).abs() <= want[2]).all()


@pytest.mark.parametrize("lens,N,G,D,q_scale", [([900], 1, 4, 128, 0.3), ([900], 1, 4, 64, 0.3), ([20000], 1, 4, 128, 1.5),
                                                ([1500, 2500], 40, 8, 128, 0.5), ([300, 60], 64, 1, 128, 0.2),
                                                ([700, 33], 20, 8, 64, 6.0)])
def test_outputs_are_as_exact_as_their_type(lens, N, G, D, q_scale):
    """bf16 outputs are off by their own rounding and nothing that shows beside
    it. Weights that count 16 bits add errors of 2^-16 of a weight, a hundredth
    of the rounding's, and fp32 sums of 20000 terms less: together below 2 % of
    the root mean square (errors that do not depend on one another add in
    squares)."""
    c = paged.Case(32, lens, N, 4, G, D, 64, "bf16", N > 1, q_scale=q_scale)
    want = c.expected()[0]
    off = sv.tree_attention(**c.args())["out"].double().cpu() - want
    rounding = want.bfloat16().double() - want
    assert off.square().mean().sqrt() <= 1.02 * rounding.square().mean().sqrt()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("octaves", [3, 10, 30, 60])
def test_values_near_the_largest(D, octaves, dtype):
    """Values of 2^100: weighted sums stay in range wherever the scores jump, in
    the middle of a tile or at its edges, since a weight is at most 2^8 before
    its row's reference follows (2^8 x 2^100 x 600 terms < 2^127)."""
    for at in (64, 130, 191, 500):
        c = paged.Case(33, [600], 4, 1, 2, D, 16, dtype, False, q_scale=0.0)
        c.q[..., 0] = 1.0
        for t in range(604):
            row = c.k[c.table[0, t // 16], t % 16, 0]
            row[0] = octaves * math.log(2.0) * D ** 0.5 if t >= at else 0.0
        c.v = (c.v.float().clamp(-4, 4) * 2.0 ** 98).to(c.v.dtype)
        got = sv.tree_attention(with_lse=True, **c.args())
        paged.assert_attention(got, c.expected(), f"jump at {at}")
