"""The paged key / value cache of a verifying target model: cases, plain forms and 64-bit results.

One verification step appends the keys and values of the drafted nodes to every
sequence's cache (``cache_append``), lets the nodes attend to the committed
context and to their ancestors (``tree_attention``), and, after verification,
moves the accepted path's entries together (``cache_compact``). Sequences share
pages (``cache_fork``) and hold or release them (``cache_resize``).

A page holds ``page_size`` tokens of one sequence; position t of sequence b is
slot t % page_size of page page_table[b, t // page_size]. ``run`` takes the plain
form (elementary torch operations in 32 bits) or, where ``own`` is true, the
library's calls.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}
# the costliest listed attention case: no drawn one is larger
MOST_BYTES, MOST_FLOPS, MOST_SCORES = 8.0e8, 1.2e11, 6.0e8


def _attention(name, B, N, kv_heads, group, D, page_size, len_lo, len_hi, dtype="bf16", tree=True):
    return dict(name=name, kind="attention", B=B, N=N, kv_heads=kv_heads, group=group, D=D, page_size=page_size,
                len_lo=len_lo, len_hi=len_hi, dtype=dtype, tree=tree)


def listed():
    return [
        # one user's step with a drafted chain of gamma = 4 tokens after the last one: the latency of a small call
        _attention("chain_b1_n5", 1, 5, 8, 4, 128, 16, 1000, 1000, tree=False),
        # plain decoding, one token a sequence, a batch of very unequal contexts
        _attention("token_b64_ragged", 64, 1, 8, 4, 128, 64, 1, 8192, tree=False),
        # draft trees of 64 nodes for 16 sequences (the tree and rest workloads), a key / value head for each query head
        _attention("tree_b16_n64_heads32", 16, 64, 32, 1, 128, 16, 150, 1900),
        # the same trees with eight query heads on each key / value head: the products bound it
        _attention("tree_b16_n64_group8", 16, 64, 8, 8, 128, 32, 300, 4000),
        # a tree over one long document, an odd node count and length
        _attention("tree_b1_n61_long", 1, 61, 8, 4, 128, 64, 100003, 100003),
        # float32 logit-exact setups: drafted chains of gamma = 7, small heads
        _attention("chain_b8_n8_f32", 8, 8, 12, 1, 64, 16, 20, 1500, dtype="f32", tree=False),
        # the drafted chains of 64 sequences written to one layer's cache
        dict(name="append_b64_n8", kind="append", B=64, N=8, kv_heads=8, D=128, page_size=16, len_lo=1, len_hi=500,
             dtype="bf16"),
        # prompt chunks written to one layer's cache, unequal lengths
        dict(name="append_b8_n1000", kind="append", B=8, N=1000, kv_heads=32, D=128, page_size=64, len_lo=0,
             len_hi=700, dtype="bf16"),
        # accepted tree paths moved together in every layer (16 sequences, depth <= 6)
        dict(name="compact_b16_l32", kind="compact", B=16, N=64, W=7, layers=32, kv_heads=8, D=128, page_size=16,
             len_lo=1, len_hi=200, dtype="bf16"),
        # long retrieved paths (depth <= 16) of a large batch, float32 caches
        dict(name="compact_b61_l12_f32", kind="compact", B=61, N=64, W=17, layers=12, kv_heads=4, D=64, page_size=32,
             len_lo=1, len_hi=120, dtype="f32"),
        # four prompts, three continuations each: the former branches released, new ones forked
        dict(name="fork_b4_x3_l8", kind="fork", B=4, copies=3, layers=8, kv_heads=8, D=128, page_size=16, len_lo=30,
             len_hi=300, spare=64, dtype="bf16"),
        # sixteen prompts, four continuations each, a deep model and a large pool
        dict(name="fork_b16_x4_l32", kind="fork", B=16, copies=4, layers=32, kv_heads=8, D=128, page_size=32,
             len_lo=100, len_hi=600, spare=300, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["attention"] * 5 + ["append", "compact", "fork"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    heads, D, ps = rng.choice([1, 2, 4, 5, 8, 12, 16, 32]), rng.choice([64, 128]), rng.choice([16, 32, 64])
    while kind == "attention":
        tree = rng.random() < 0.6
        c = dict(kind=kind, B=_log_int(rng, 1, 64), N=_log_int(rng, 2, 500) if tree else _log_int(rng, 1, 16),
                 kv_heads=heads, group=rng.choice([1, 1, 2, 3, 4, 7, 8]), D=D, page_size=ps, len_lo=0,
                 len_hi=_log_int(rng, 1, 100000), dtype=dtype, tree=tree)
        c["len_lo"] = int(c["len_hi"] * rng.random() ** 2)
        w = _bounds(c)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS / (1 if dtype == "bf16" else 16) \
                and w["scores"] <= MOST_SCORES:
            return c
        heads = rng.choice([1, 2, 4, 5, 8, 12, 16, 32])
    if kind == "append":
        return dict(kind=kind, B=_log_int(rng, 1, 64), N=_log_int(rng, 1, 1000), kv_heads=rng.choice([1, 2, 5, 8]), D=D,
                    page_size=ps, len_lo=0, len_hi=_log_int(rng, 1, 700), dtype=dtype)
    if kind == "compact":
        return dict(kind=kind, B=_log_int(rng, 1, 61), N=_log_int(rng, 20, 200), W=rng.randint(2, 17),
                    layers=_log_int(rng, 1, 32), kv_heads=rng.choice([1, 2, 4, 5]), D=D, page_size=ps, len_lo=0,
                    len_hi=_log_int(rng, 1, 150), dtype=dtype)
    return dict(kind=kind, B=_log_int(rng, 1, 16), copies=rng.randint(1, 4), layers=_log_int(rng, 1, 24),
                kv_heads=rng.choice([1, 2, 4, 5]), D=D, page_size=ps, len_lo=1, len_hi=_log_int(rng, 2, 600),
                spare=_log_int(rng, 1, 300), dtype=dtype)


def _bounds(c):
    """Upper bounds of an attention case's bytes, operations and plain-form scores."""
    T = c["len_hi"] + c["N"]
    rows = c["B"] * c["N"] * c["kv_heads"] * c["group"]
    return dict(bytes=2.0 * c["B"] * T * c["kv_heads"] * c["D"] * ESIZE[c["dtype"]] + 2.0 * rows * c["D"] * 4,
                flops=4.0 * rows * c["D"] * T, scores=float(rows) * T)


def _lengths(case):
    """Context lengths: evenly spread over the case's range in a fixed shuffled order (the same for every seed, so
    that work() is exact), both ends included."""
    B, lo, hi = case["B"], case["len_lo"], case["len_hi"]
    if B == 1:
        return np.array([hi], np.int64)
    x = lo + (np.arange(B) * (hi - lo)) // (B - 1)
    return x[np.random.RandomState(B).permutation(B)]


def _counts(case):
    """Nodes of each sequence: most have all N, every fourth has fewer."""
    B, N = case["B"], case["N"]
    return np.where(np.arange(B) % 4 == 3, max(1, (2 * N) // 3), N)


def _trees(case, seed):
    """Breadth-first draft trees: parents [B, N] and the ancestor masks [B, N, N] (zero rows and columns from a
    sequence's node count on)."""
    B, N = case["B"], case["N"]
    rng = np.random.default_rng([seed, 5])
    parent = np.full((B, N), -1, np.int64)
    mask = np.zeros((B, N, N), np.uint8)
    mask[:, 0, 0] = 1
    rows = np.arange(B)
    for i in range(1, N):  # a parent among the latest nodes, never before its predecessor's: breadth-first order
        lo = np.maximum(parent[:, i - 1], (i - 1) // 4)
        parent[:, i] = rng.integers(lo, np.minimum(i, lo + 3))
        mask[:, i] = mask[rows, parent[:, i]]
        mask[:, i, i] = 1
    mask *= (np.arange(N)[None, :] < _counts(case)[:, None])[:, :, None].astype(np.uint8)
    return parent, mask


def _pool(case, tokens, seed, layers, spare=3):
    """Caches [layers, pages, page_size, heads, D] and a page table for sequences of `tokens` positions, pages in
    random order; table entries past a sequence's end are -1."""
    ps = case["page_size"]
    need = -(-np.asarray(tokens) // ps)
    M = int(max(1, need.max()))
    total = int(need.sum())
    P = total + spare
    order = np.random.default_rng([seed, 7]).permutation(P)[:total]
    table = np.full((len(need), M), -1, np.int32)
    table[np.arange(M)[None, :] < need[:, None]] = order
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (layers, P, ps, case["kv_heads"], case["D"])
    td = DTYPES[case["dtype"]]
    k = torch.empty(shape, dtype=td, device="cuda").normal_(generator=g)
    v = torch.empty(shape, dtype=td, device="cuda").normal_(generator=g)
    return k, v, torch.from_numpy(table).cuda(), need, g


def prepare(case, seed):
    kind, td = case["kind"], DTYPES[case["dtype"]]
    lens = _lengths(case)
    s = dict(kind=kind, page_size=case["page_size"], cache_len=torch.from_numpy(lens.astype(np.int32)).cuda())
    if kind in ("attention", "append"):
        B, N, D = case["B"], case["N"], case["D"]
        n = _counts(case)
        s["n_nodes"] = torch.from_numpy(n.astype(np.int32)).cuda()
        k, v, s["page_table"], _, g = _pool(case, lens + n, seed, 1)
        s["k_cache"], s["v_cache"] = k[0], v[0]
        if kind == "attention":
            q = torch.randn(B, N, case["kv_heads"] * case["group"], D, generator=g, device="cuda")
            s["q"] = (1.5 * q).to(td)
            s["mask"] = torch.from_numpy(_trees(case, seed)[1]).cuda() if case["tree"] else None
        else:
            s["k"] = torch.randn(B, N, case["kv_heads"], D, generator=g, device="cuda").to(td)
            s["v"] = torch.randn(B, N, case["kv_heads"], D, generator=g, device="cuda").to(td)
        return s
    if kind == "compact":
        B, N, W = case["B"], case["N"], case["W"]
        rng = np.random.default_rng([seed, 9])
        accept = np.arange(B) % W
        path = np.full((B, W), -1, np.int32)
        for b in range(B):
            a = min(int(accept[b]), N - 1)
            accept[b] = a
            path[b, 0] = 0
            path[b, 1:a + 1] = np.sort(rng.choice(np.arange(1, N), size=a, replace=False))
        s["k_cache"], s["v_cache"], s["page_table"], _, _ = _pool(case, lens + N, seed, case["layers"])
        s["path"] = torch.from_numpy(path).cuda()
        s["accept"] = torch.from_numpy(accept.astype(np.int32)).cuda()
        return s
    # fork: rows 0..B-1 of the table hold the prompts, the rows after them their continuations (empty at the start)
    B, C = case["B"], case["copies"]
    k, v, table, need, _ = _pool(case, lens, seed, case["layers"], spare=B * C + case["spare"])
    M = table.shape[1]
    refs = torch.zeros(k.shape[1], dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    s["k_cache"], s["v_cache"], s["page_refs"] = k, v, refs
    s["page_table"] = torch.cat([table, torch.full((B * C, M), -1, dtype=torch.int32, device="cuda")])
    s["cache_len"] = torch.cat([s["cache_len"], torch.zeros(B * C, dtype=torch.int32, device="cuda")])
    s["src"] = torch.arange(B * C, dtype=torch.int32, device="cuda") // C
    s["dst"] = torch.arange(B, B + B * C, dtype=torch.int32, device="cuda")
    s["none"] = torch.zeros(B * C, dtype=torch.int32, device="cuda")
    return s


def _plain_attention(s):
    q, table, ps = s["q"], s["page_table"].long().clamp(min=0), s["page_size"]
    B, N, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    G, T = Hq // Hkv, table.shape[1] * ps
    keys = s["k_cache"][table].reshape(B, T, Hkv, D).float()
    values = s["v_cache"][table].reshape(B, T, Hkv, D).float()
    node = torch.arange(T, device=q.device)[None, :] - s["cache_len"].long()[:, None]     # [B, T]: < 0 context
    count = s["n_nodes"].long()[:, None]
    row = torch.arange(N, device=q.device)
    inside = ((node >= 0) & (node < count))[:, None, :]
    j = node.clamp(0, N - 1)
    if s["mask"] is not None:
        seen = s["mask"].gather(2, j[:, None, :].expand(B, N, T)).bool()
    else:
        seen = j[:, None, :] <= row[None, :, None]
    allowed = ((node < 0)[:, None, :] | (inside & seen)) & (row[None, :] < count)[:, :, None]      # [B, N, T]
    x = q.float().reshape(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    score = (x @ keys.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    score = score.reshape(B, Hkv, N, G, T).masked_fill_(~allowed[:, None, :, None, :], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    p = (score - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    values = values * (node < count)[:, :, None, None]
    o = p.reshape(B, Hkv, N * G, T) @ values.permute(0, 2, 1, 3)
    o = o.reshape(B, Hkv, N, G, D) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log()).squeeze(-1)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(q.dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, N, Hq)}


def _slots(s, position):
    """Row of the flattened [pages * page_size] cache that holds each sequence's position."""
    ps = s["page_size"]
    return s["page_table"].long().gather(1, position // ps) * ps + position % ps


def _plain_append(s):
    B, N = s["k"].shape[:2]
    i = torch.arange(N, device=s["k"].device)[None, :].expand(B, N)
    i = torch.where(i < s["n_nodes"].long()[:, None], i, torch.zeros_like(i))  # padding repeats node 0
    at = _slots(s, s["cache_len"].long()[:, None] + i)
    pick = i[:, :, None, None].expand(B, N, *s["k"].shape[2:])
    for new, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        cache.view(-1, *cache.shape[2:])[at] = new.gather(1, pick)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_compact(s):
    B, W = s["path"].shape
    i = torch.arange(W, device=s["path"].device)[None, :].expand(B, W)
    i = torch.where(i <= s["accept"].long()[:, None], i, torch.zeros_like(i))  # past the path: node 0 onto itself
    start = s["cache_len"].long()[:, None]
    to, frm = _slots(s, start + i), _slots(s, start + s["path"].long().gather(1, i))
    for cache in (s["k_cache"], s["v_cache"]):
        flat = cache.view(cache.shape[0], -1, *cache.shape[3:])
        flat[:, to] = flat[:, frm]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "cache_len": s["cache_len"] + s["accept"] + 1}


def _plain_fork(s):
    table, refs, ps = s["page_table"], s["page_refs"], s["page_size"]
    src, dst = s["src"].long(), s["dst"].long()
    # the former branches: one reference less for every page that they hold
    held = table[dst].long()
    refs.index_add_(0, held.clamp(min=0).reshape(-1), -(held >= 0).reshape(-1).to(torch.int32))
    # shared: every full page; the page that is partly filled is copied into the lowest free one
    length = s["cache_len"][src].long()
    full, rest = length // ps, length % ps
    F, M = held.shape
    col = torch.arange(M, device=table.device)[None, :]
    mine = table[src].long()
    shared = col < full[:, None]
    refs.index_add_(0, mine.clamp(min=0).reshape(-1), shared.reshape(-1).to(torch.int32))
    free = torch.sort((refs > 0).to(torch.int32), stable=True).indices
    rank = (rest > 0).long().cumsum(0) - 1
    fresh = free[rank.clamp(min=0)]
    partial = (col == full[:, None]) & (rest > 0)[:, None]
    table[dst] = torch.where(shared, mine, torch.where(partial, fresh[:, None], torch.full_like(mine, -1))).to(torch.int32)
    refs.index_add_(0, fresh, (rest > 0).to(torch.int32))
    s["cache_len"][dst] = length.to(torch.int32)
    # slots past the copied ones repeat slot 0; with nothing to copy, the prompt's first row goes onto itself
    some = rest > 0
    first = mine[:, 0]
    old = torch.where(some, mine.gather(1, full.clamp(max=M - 1)[:, None]).squeeze(1), first)
    new = torch.where(some, fresh, first)
    slot = torch.arange(ps, device=table.device)[None, :].expand(F, ps)
    slot = torch.where(slot < rest[:, None], slot, torch.zeros_like(slot))
    frm, to = old[:, None] * ps + slot, new[:, None] * ps + slot
    for cache in (s["k_cache"], s["v_cache"]):
        flat = cache.view(cache.shape[0], -1, *cache.shape[3:])
        flat[:, to] = flat[:, frm]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "page_table": table, "page_refs": refs,
            "cache_len": s["cache_len"]}


def _own(s):
    import speculative_decoding_verification_05_gb300 as sv

    kind = s["kind"]
    if kind == "attention":
        r = sv.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cache_len"], mask=s["mask"],
                              n_nodes=s["n_nodes"], with_lse=True)
        return {"out": r["out"], "lse": r["lse"]}
    if kind == "append":
        sv.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["cache_len"],
                        n_nodes=s["n_nodes"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if kind == "compact":
        r = sv.cache_compact(s["k_cache"], s["v_cache"], s["page_table"], s["cache_len"], s["accept"], s["path"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "cache_len": r["cache_len"]}
    sv.cache_resize(s["page_table"], s["page_refs"], s["dst"], s["none"], s["page_size"])
    sv.cache_fork(s["k_cache"], s["v_cache"], s["page_table"], s["cache_len"], s["page_refs"], s["src"], s["dst"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "page_table": s["page_table"],
            "page_refs": s["page_refs"], "cache_len": s["cache_len"]}


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "append": _plain_append, "compact": _plain_compact,
            "fork": _plain_fork}[state["kind"]](state)


def work(case):
    es, D, H, ps = ESIZE[case["dtype"]], case["D"], case["kv_heads"], case["page_size"]
    lens = _lengths(case)
    if case["kind"] == "attention":
        n, G, N = _counts(case), case["group"], case["N"]
        rows = case["B"] * N * H * G
        real = float((n * (lens + n)).sum()) * H * G
        # keys and values once, queries, outputs, log-sums, the mask, tables and lengths
        bytes_ = (2.0 * float((lens + n).sum()) * H * D + 2.0 * rows * D) * es + 4.0 * rows
        bytes_ += float((n * n).sum()) if case["tree"] else 0.0
        return {"bytes": bytes_ + 4.0 * float((-(-(lens + n) // ps)).sum()) + 8.0 * case["B"], "flops": 4.0 * D * real}
    if case["kind"] == "append":
        return {"bytes": 4.0 * float(_counts(case).sum()) * H * D * es, "flops": 0.0}
    if case["kind"] == "compact":
        moved = float(np.minimum(np.arange(case["B"]) % case["W"], case["N"] - 1).sum())
        return {"bytes": max(4.0 * moved * case["layers"] * H * D * es, 64.0 * case["B"]), "flops": 0.0}
    rest, full = lens % ps, lens // ps
    return {"bytes": case["copies"] * (4.0 * float(rest.sum()) * case["layers"] * H * D * es
                                       + 16.0 * float((full + 1).sum())), "flops": 0.0}


def exact(case, seed):
    """Attention from its definition, one sequence at a time, in 64 bits; what the other operators return is moved
    or counted, not computed."""
    if case["kind"] != "attention":
        return None
    s = prepare(case, seed)
    lens, counts = _lengths(case), _counts(case)
    B, N, H, G, D = case["B"], case["N"], case["kv_heads"], case["group"], case["D"]
    out = torch.zeros(B, N, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, H * G), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        L, n = int(lens[b]), int(counts[b])
        pages = s["page_table"][b][:-(-(L + n) // case["page_size"])].long()
        keys = s["k_cache"][pages].flatten(0, 1)[:L + n]
        values = s["v_cache"][pages].flatten(0, 1)[:L + n]
        see = torch.ones(n, L + n, dtype=torch.bool, device="cuda")
        see[:, L:] = s["mask"][b, :n, :n].bool() if s["mask"] is not None else see[:, L:].tril()
        for h in range(H):
            x = s["q"][b, :n, h * G:(h + 1) * G].double()                        # [n, G, D]
            z = torch.einsum("ngd,td->gnt", x, keys[:, h].double()) / math.sqrt(D)
            z = torch.where(see, z, torch.full_like(z, -math.inf))
            lse[b, :n, h * G:(h + 1) * G] = torch.logsumexp(z, dim=-1).transpose(0, 1)
            out[b, :n, h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", torch.softmax(z, dim=-1),
                                                         values[:, h].double())
    return {"out": out, "lse": lse}
