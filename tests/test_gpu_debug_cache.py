"""The cache's operators and the log probabilities through the debug build: no index check fails,
and every result is the release build's."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_05_gb300 as sv

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def steps(td, D, G, ps, interleaved, dim, wide):
    """Two steps of a bounded cache with forks; every tensor that they leave."""
    layers, B, H, N, V, width = 2, 4, 3, 9, 700, 64 // ps + 3
    g = torch.Generator(device="cuda").manual_seed(D + G)
    shape = (layers, 3 * B * width, ps, H + wide, D + 16 * wide)
    kc, vc = (torch.zeros(shape, dtype=td, device="cuda")[..., :H, :D] for _ in range(2))
    table = torch.full((B + 1, width), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(shape[1], dtype=torch.int32, device="cuda")
    weights = torch.rand(layers, B, H, width * ps, generator=g, device="cuda")
    length = i32([5, 0, 37, 60])
    out = [sv.cache_resize(table, refs, i32(range(B)), length, ps)["status"]]
    for step in range(2):
        n = i32([N, 3, 0, N - 1])
        out.append(sv.cache_resize(table, refs, i32(range(B)), length.clamp(min=0) + N, ps)["status"])
        mine = table[:B].contiguous()
        for y in range(layers):
            q, k, v = (torch.randn(B, N, h, D, generator=g, device="cuda").to(td) for h in (H * G, H, H))
            r = sv.cache_append_rotary(q, k, v, kc[y], vc[y], mine, length, sv.rotary(dim, interleaved=interleaved),
                                       positions=length + 100, n_nodes=n, page_refs=refs)
            o = sv.tree_attention(r["q"], kc[y], vc[y], mine, length, n_nodes=n, with_lse=True)
            s = sv.cache_weigh(r["q"], o["lse"], kc[y], mine, length, weights[y], accept_len=n - 1)
            out += [*r.values(), *o.values(), *s.values()]
        acc = (n - 1).clamp(min=0)
        path = torch.tensor([[0, 2, 3, 5, 8]] * B, dtype=torch.int32, device="cuda")
        c = sv.cache_compact(kc, vc, mine, length, i32([4, 1, 0, 3]), path, page_refs=refs)
        e = sv.cache_evict(kc, vc, mine, c["cache_len"], weights, 40, sink=3, recent=7, page_refs=refs)
        length = e["cache_len"].clamp(min=0)
        out += [*c.values(), *e.values(), acc, weights.clone()]
        z = torch.randn(B, N, V, generator=g, device="cuda").to(td)
        t = torch.randint(-1, V, (B, N), generator=g, device="cuda", dtype=torch.int32)
        z[1, 2] = torch.nan
        out += [*sv.token_logprobs(z, t, top=7).values()]
    lens5 = torch.cat([length, i32([0])])
    f = sv.cache_fork(kc, vc, table, lens5, refs, i32([3]), i32([4]))
    return out + [*f.values(), lens5, kc.clone(), vc.clone(), table, refs]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,G,ps,interleaved,dim,wide", [(64, 2, 8, False, 64, 0), (128, 4, 16, True, 100, 1),
                                                         (96, 1, 8, False, 20, 0), (40, 3, 16, False, 40, 1)])
def test_a_bounded_cache(dtype, D, G, ps, interleaved, dim, wide):
    args = (dtype, D, G, ps, interleaved, dim, wide)
    want = steps(*args)
    lib = sv.load_library(sv.DEBUG_LIB_PATH)
    with sv.use_library(sv.DEBUG_LIB_PATH):
        got = steps(*args)
    torch.cuda.synchronize()
    assert lib.spec_debug_failures(None) == 0
    for i, (a, b) in enumerate(zip(want, got)):
        assert torch.equal(a.nan_to_num(3.0) if a.is_floating_point() else a, b.nan_to_num(3.0) if b.is_floating_point() else b), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,P,V,top", [(2, 2, 70001, 32), (700, 1, 2049, 5), (3, 1, 31, 31)])
def test_log_probabilities(dtype, B, P, V, top):
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(B, P, V, generator=g, device="cuda").to(dtype)
    z[0, 0] = 1.0
    z[1, 0, V // 3:] = torch.nan
    t = torch.randint(-1, V, (B, P), generator=g, device="cuda", dtype=torch.int32)
    want = sv.token_logprobs(z, t, top=top)
    lib = sv.load_library(sv.DEBUG_LIB_PATH)
    with sv.use_library(sv.DEBUG_LIB_PATH):
        got = sv.token_logprobs(z, t, top=top)
    torch.cuda.synchronize()
    assert lib.spec_debug_failures(None) == 0
    for k in want:
        assert torch.equal(want[k].nan_to_num(3.0), got[k].nan_to_num(3.0)) if want[k].is_floating_point() else torch.equal(want[k], got[k]), k
