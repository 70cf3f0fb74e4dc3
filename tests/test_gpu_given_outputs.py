"""Outputs that the caller passes: used where they fit, refused where they do not."""

import pytest
import torch

import paged
import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu


def test_attention_outputs():
    c = paged.Case(51, [70, 9], 6, 2, 4, 128, 16, "bf16", True)
    a = c.args()
    want = sv.tree_attention(with_lse=True, **a)
    good = dict(out=torch.empty_like(a["q"]), lse=torch.empty(2, 6, 8, device="cuda"),
                status=torch.empty(2, dtype=torch.int32, device="cuda"))
    got = sv.tree_attention(out=good, **a)
    for k in good:
        assert got[k] is good[k] and torch.equal(got[k], want[k])
    for key, bad in (("out", good["out"][:1]), ("out", good["out"].float()), ("out", good["out"].cpu()),
                     ("out", torch.empty(2, 6, 8, 256, dtype=torch.bfloat16, device="cuda")[..., :128]),
                     ("lse", good["lse"][:, :5]), ("lse", good["lse"].double()), ("lse", good["lse"].cpu()),
                     ("status", good["status"].long()), ("status", good["status"][:1]), ("status", good["status"].cpu())):
        with pytest.raises(sv.SpecError):
            sv.tree_attention(out={**good, key: bad}, **a)


def test_verify_outputs():
    z = torch.randn(3, 5, 1000, device="cuda")
    d, t = torch.randn(3, 4, 1000, device="cuda"), torch.randint(1000, (3, 4), dtype=torch.int32, device="cuda")
    want = sv.verify(z, d, t, debug=True)
    good = {k: torch.empty_like(v) for k, v in want.items()}
    got = sv.verify(z, d, t, out=good)
    for k in good:
        assert got[k] is good[k] and torch.equal(got[k], want[k])
    for key, bad in (("accepted", good["accepted"].long()), ("tokens", good["tokens"][:, :4]),
                     ("tokens", torch.empty(3, 10, dtype=torch.int32, device="cuda")[:, ::2]),
                     ("next_token", good["next_token"].cpu()), ("status", good["status"][:2]),
                     ("probs", good["probs"].double())):
        with pytest.raises(sv.SpecError):
            sv.verify(z, d, t, out={**good, key: bad})
