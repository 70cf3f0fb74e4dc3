"""The operators of a verification step in a bounded cache together, as a server
runs them: rotary append, attention, verification, log probabilities, the
accepted path kept, its rows weighed, positions evicted, pages released - step
after step, against lists of entries in 64 bits.

Tolerances: as in the operators' own tests; the lists take over the cache's bits
after they were compared, so that nothing adds up over the steps.
"""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv
from test_gpu_rotary import angles, rotated

pytestmark = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype,D,G,interleaved", [("bf16", 64, 2, False), ("bf16", 128, 4, True), ("f32", 64, 1, False),
                                                   ("bf16", 96, 2, False)])
def test_steps(dtype, D, G, interleaved):
    B, layers, H, N, V, ps, budget, sink, recent, width = 3, 2, 2, 12, 120, 8, 11, 2, 4, 4
    td, half = TD[dtype], 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    rng, g = np.random.default_rng(D + G), torch.Generator().manual_seed(D + G)
    kc, vc = (torch.zeros(layers, B * width, ps, H, D, dtype=td, device="cuda") for _ in range(2))
    table, refs = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), torch.zeros(B * width, dtype=torch.int32, device="cuda")
    weights = torch.zeros(layers, B, H, width * ps, device="cuda")
    length, text = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    rot = sv.rotary(D // 2, interleaved=interleaved, scaling="linear", scale=2.0)
    # the lists: keys, values [layers][B][H] and weights of what each head holds
    K, W = ([[[[] for _ in range(H)] for _ in range(B)] for _ in range(layers)] for _ in range(2))
    evicted = 0
    for step in range(12):
        # draft trees of random continuations
        cand = torch.from_numpy(rng.integers(0, 4, (B, 6, 4))).int().cuda()
        root = i32(rng.integers(0, 4, B))
        t = sv.tree_build(cand, root, V, N)
        n = t["n_nodes"]
        assert sv.cache_resize(table, refs, None, length + n, ps)["status"].sum() == 0
        q = [torch.randn(B, N, H * G, D, generator=g).to(td) for _ in range(layers)]
        k, v = ([torch.randn(B, N, H, D, generator=g).to(td) for _ in range(layers)] for _ in range(2))
        lse, turned = [], []
        for y in range(layers):
            r = sv.cache_append_rotary(q[y].cuda(), k[y].cuda(), v[y].cuda(), kc[y], vc[y], table, length, rot, positions=text,
                                       depth=t["depth"], n_nodes=n, page_refs=refs)
            assert r["status"].sum() == 0
            turned.append(r["q"])
            o = sv.tree_attention(r["q"], kc[y], vc[y], table, length, t["mask"], n, with_lse=True)
            assert o["status"].sum() == 0
            lse.append(o["lse"])
        # logits under which some drafted nodes are accepted
        z = torch.randn(B, N, V, generator=g).cuda()
        z[:, :, :4] += 2.5
        unused = torch.arange(N, device="cuda") >= n[:, None]
        tok, par, dep = (torch.where(unused, t[x][:, 1:2], t[x]) for x in ("node_tokens", "parent", "depth"))
        res = sv.verify_tree(z, tok, par, dep, 4)
        acc, path = res["accept_len"], res["path_nodes"]
        # the emitted tokens' log probabilities, from their parents' rows
        rows = z.gather(1, path.clamp(min=0).long()[..., None].expand(-1, -1, V))
        lp = sv.token_logprobs(rows, res["tokens"], top=2)
        ref = torch.log_softmax(rows.double(), -1)
        for b in range(B):
            for i in range(5):
                x = int(res["tokens"][b, i])
                want = float(ref[b, i, x]) if x >= 0 else 0.0
                assert abs(float(lp["logprob"][b, i]) - want) <= 2.0 ** -15
                if x >= 0:
                    assert lp["rank"][b, i] == 0 and lp["top_tokens"][b, i, 0] == x   # (greedy: the likeliest)
        kept = sv.cache_compact(kc, vc, table, length, acc, path, refs)
        assert kept["status"].sum() == 0
        for y in range(layers):
            s = sv.cache_weigh(turned[y], lse[y], kc[y], table, length, weights[y], acc, path)
            assert s["status"].sum() == 0
        # the same on the lists
        tab, L = table.cpu().numpy(), length.tolist()
        at = lambda b, p: (int(tab[b, p // ps]), p % ps)
        for y in range(layers):
            kk = kc[y].cpu()
            for b in range(B):
                nodes = path[b, :int(acc[b]) + 1].tolist()
                pos = [int(text[b]) + int(t["depth"][b, i]) for i in nodes]
                want, size = rotated(k[y][b, nodes].double(), angles(rot, pos), D // 2, interleaved, 1.0)
                for h in range(H):
                    old = torch.stack([kk[at(b, p)][h] for p in range(L[b])]) if L[b] else torch.zeros(0, D, dtype=td)
                    assert torch.equal(old, torch.stack(K[y][b][h]) if L[b] else old)
                    for r, i in enumerate(nodes):
                        new = kk[at(b, L[b] + r)][h]
                        assert ((new.double() - want[r, h]).abs() <= 2.0 ** -21 * size[r, h] + half * want[r, h].abs()).all()
                        K[y][b][h].append(new)
                        W[y][b][h].append(0.0)
                    keys = torch.stack(K[y][b][h]).double()
                    x = turned[y][b, nodes].double().cpu()[:, h * G:(h + 1) * G]
                    s = torch.einsum("rgd,td->rgt", x, keys) * D ** -0.5
                    size_s = torch.einsum("rgd,td->rgt", x.abs(), keys.abs()) * D ** -0.5
                    see = torch.arange(len(keys))[None] <= L[b] + torch.arange(len(nodes))[:, None]
                    s = s.masked_fill(~see[:, None], -math.inf)
                    p = torch.softmax(s, -1)
                    # (the log-sum is the attention's own: off by as much as a score and its sum)
                    rel = (D + 8) * 2.0 ** -22 * size_s.amax() + 2.0 ** -20
                    got = weights[y, b, h, :len(keys)].double().cpu()
                    exp = torch.tensor(W[y][b][h], dtype=torch.float64) + p.sum((0, 1))
                    assert ((got - exp).abs() <= rel * p.sum((0, 1)) + 2.0 ** -23 * exp).all()
                    W[y][b][h] = got.tolist()
        text = text + acc + 1
        length = kept["cache_len"]
        # the cache is bounded
        e = sv.cache_evict(kc, vc, table, length, weights, budget, sink, recent, refs)
        assert e["status"].sum() == 0
        for b in range(B):
            now = int(length[b])
            if now > budget:
                evicted += 1
                for y in range(layers):
                    for h in range(H):
                        mid = sorted(range(sink, now - recent), key=lambda i: (-W[y][b][h][i], i))[:budget - sink - recent]
                        keep = list(range(sink)) + sorted(mid) + list(range(now - recent, now))
                        K[y][b][h], W[y][b][h] = ([x[y][b][h][i] for i in keep] for x in (K, W))
        length = e["cache_len"]
        assert length.tolist() == [len(K[0][b][0]) for b in range(B)]
        assert sv.cache_resize(table, refs, None, length, ps)["status"].sum() == 0
        assert int(refs.sum()) == sum(-(-x // ps) for x in length.tolist())
        for y in range(layers):
            for b in range(B):
                for h in range(H):
                    assert weights[y, b, h].tolist()[:len(W[y][b][h])] == W[y][b][h] and (weights[y, b, h, len(W[y][b][h]):] == 0).all()
    assert evicted > 0 and (text > length).any()
