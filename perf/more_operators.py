"""A verification step with positions of its own and a bounded cache: cases, plain forms and 64-bit results.

One layer's drafted nodes get rotary positions and are written to the paged
cache in one call (``cache_append_rotary``; a node's text position is not its
place in the cache once tokens were evicted, and is its depth's in a tree). After
verification the accepted tokens' log probabilities are reported
(``token_logprobs``), the accepted rows' attention weights are added up for every
cached position and key / value head (``cache_weigh``), and from time to time the
positions of the least weight leave the cache (``cache_evict``).

``run`` takes the plain form (elementary torch operations, in 32 bits; angles in
64) or, where ``own`` is true, the library's calls.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}
# the costliest listed cases: no drawn one is larger
MOST_LOGITS, MOST_MOVED, MOST_KEYS, MOST_SCORES = 2.6e8, 1.5e8, 5.5e8, 1.4e8
MOST_EVICT = 4.5e9


def _logprobs(name, B, P, V, dtype, top, temperature=1.0, step=True):
    return dict(name=name, kind="logprobs", B=B, P=P, V=V, dtype=dtype, top=top, temperature=temperature, step=step)


def _rotary(name, B, N, heads, kv_heads, D, dim, page_size, len_lo, len_hi, dtype, interleaved=False, tree=False,
            scaling="none", shift=0):
    return dict(name=name, kind="rotary", B=B, N=N, heads=heads, kv_heads=kv_heads, D=D, dim=dim, page_size=page_size,
                len_lo=len_lo, len_hi=len_hi, dtype=dtype, interleaved=interleaved, tree=tree, scaling=scaling,
                shift=shift)


def _weigh(name, B, N, W, kv_heads, group, D, page_size, len_lo, len_hi, dtype):
    return dict(name=name, kind="weigh", B=B, N=N, W=W, kv_heads=kv_heads, group=group, D=D, page_size=page_size,
                len_lo=len_lo, len_hi=len_hi, dtype=dtype)


def _evict(name, B, layers, kv_heads, D, page_size, len_lo, len_hi, budget, sink, recent, dtype):
    return dict(name=name, kind="evict", B=B, layers=layers, kv_heads=kv_heads, D=D, page_size=page_size,
                len_lo=len_lo, len_hi=len_hi, budget=budget, sink=sink, recent=recent, dtype=dtype)


def listed():
    return [
        # one user's step with a drafted chain of gamma = 4: the latency of a small call
        _logprobs("logprobs_b1_p5", 1, 5, 32000, "bf16", 5),
        # a large-vocabulary step of 64 sequences; the rows after a rejection carry no token
        _logprobs("logprobs_b64_p8", 64, 8, 128256, "f32", 20, temperature=0.8),
        # scoring two prompts, no alternatives asked for
        _logprobs("logprobs_prompts", 2, 1000, 32016, "bf16", 0, step=False),
        # one user's drafted chain, one layer
        _rotary("rotary_b1_n5", 1, 5, 32, 8, 128, 128, 16, 1000, 1000, "bf16"),
        # prompt chunks of eight sequences, one layer, a long-context model
        _rotary("rotary_b8_n1000", 8, 1000, 32, 8, 128, 128, 64, 0, 700, "bf16", scaling="yarn"),
        # draft trees far into a text whose cache is bounded, half of a head rotated, neighbouring pairs
        _rotary("rotary_tree_f32", 16, 61, 12, 12, 64, 32, 16, 150, 1900, "f32", interleaved=True, tree=True,
                scaling="linear", shift=500000),
        # plain decoding, one token a sequence, a batch of very unequal contexts
        _weigh("weigh_b64_token", 64, 1, 1, 8, 4, 128, 64, 1, 8192, "bf16"),
        # accepted tree paths (depth <= 6) of trees of 64 nodes, eight query heads on each key / value head
        _weigh("weigh_b16_path", 16, 64, 7, 8, 8, 128, 32, 300, 4000, "bf16"),
        # a prompt's last chunk over the chunks before it
        _weigh("weigh_prompt", 1, 500, 500, 8, 4, 128, 16, 4000, 4000, "bf16"),
        # float32 setups: drafted chains of gamma = 7, small heads
        _weigh("weigh_b8_f32", 8, 8, 8, 12, 1, 64, 16, 20, 1500, "f32"),
        # one sequence over its budget in a small model, odd sizes
        _evict("evict_b1_l12", 1, 12, 4, 64, 16, 1501, 1501, 1003, 4, 250, "f32"),
        # a batch in a deep model
        _evict("evict_b16_l32", 16, 32, 8, 128, 32, 1500, 4000, 1600, 4, 512, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["logprobs", "logprobs", "rotary", "rotary", "weigh", "weigh", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    while True:
        if kind == "logprobs":
            step = rng.random() < 0.7
            c = dict(kind=kind, B=_log_int(rng, 1, 64), P=rng.randint(1, 17) if step else _log_int(rng, 1, 1000),
                     V=_log_int(rng, 1000, 200000), dtype=dtype, top=rng.choice([0, 1, 5, 8, 20, 32]),
                     temperature=rng.choice([1.0, 1.0, 0.7, 1.3]), step=step)
            if c["B"] * c["P"] * c["V"] * ESIZE[dtype] <= MOST_LOGITS:
                return c
            continue
        heads, D, ps = rng.choice([1, 2, 4, 5, 8, 12, 16]), rng.choice([64, 96, 128]), rng.choice([16, 32, 64])
        group = rng.choice([1, 1, 2, 3, 4, 7, 8])
        hi = _log_int(rng, 1, 60000 if kind == "weigh" else 4000)
        lo = int(hi * rng.random() ** 2)
        if kind == "rotary":
            tree = rng.random() < 0.5
            c = dict(kind=kind, B=_log_int(rng, 1, 64), N=_log_int(rng, 1, 200 if tree else 1000), heads=heads * group,
                     kv_heads=heads, D=D, dim=rng.choice([D, D, D // 2, 24]), page_size=ps, len_lo=lo, len_hi=hi,
                     dtype=dtype, interleaved=rng.random() < 0.4, tree=tree,
                     scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]), shift=rng.choice([0, 777, 1000000]))
            if 2.0 * c["B"] * c["N"] * heads * (group + 2) * D * ESIZE[dtype] <= MOST_MOVED:
                return c
        elif kind == "weigh":
            N = rng.choice([1, _log_int(rng, 2, 17), _log_int(rng, 18, 500)])
            W = N if rng.random() < 0.5 else min(N, rng.randint(1, 17))
            c = dict(kind=kind, B=_log_int(rng, 1, 64), N=N, W=W, kv_heads=heads, group=group, D=D, page_size=ps,
                     len_lo=lo, len_hi=hi, dtype=dtype)
            keys = float(c["B"]) * (hi + N) * heads
            if keys * D * ESIZE[dtype] <= MOST_KEYS and keys * W * group <= MOST_SCORES / (1 if dtype == "bf16" else 8):
                return c
        else:
            recent, sink = rng.randint(0, hi // 3), rng.randint(0, 8)
            c = dict(kind=kind, B=_log_int(rng, 1, 16), layers=_log_int(rng, 1, 32), kv_heads=heads, D=D, page_size=ps,
                     len_lo=lo, len_hi=hi, budget=min(sink + recent + _log_int(rng, 1, max(1, hi // 2)), hi), sink=sink,
                     recent=recent, dtype=dtype)
            c["budget"] = max(c["budget"], sink + recent)
            if 2.0 * c["B"] * c["layers"] * hi * heads * D * ESIZE[dtype] <= MOST_EVICT:
                return c


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


def _rows(case):
    """Rows (nodes) of each sequence that are weighed: its whole chain, or a path of any length up to W."""
    B, W = case["B"], case["W"]
    return np.full(B, W) if W == case["N"] else 1 + np.arange(B) % W


def _asked(case):
    """Rows of each sequence that carry a token: all of them, or a step's accepted ones and the one after."""
    B, P = case["B"], case["P"]
    return 1 + (5 * np.arange(B) + P - 1) % P if case["step"] else np.full(B, P)


def _pool(case, tokens, g, seed, layers, spare=3):
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
    shape = (layers, P, ps, case["kv_heads"], case["D"])
    td = DTYPES[case["dtype"]]
    k = torch.empty(shape, dtype=td, device="cuda").normal_(generator=g)
    v = torch.empty(shape, dtype=td, device="cuda").normal_(generator=g)
    return k, v, torch.from_numpy(table).cuda()


SCALINGS = {"none": {}, "linear": dict(scaling="linear", scale=4.0), "ntk": dict(scaling="ntk", scale=8.0),
            "yarn": dict(scaling="yarn", scale=16.0, original=4096), "bands": dict(scaling="bands", scale=8.0, original=8192)}


def _frequencies(case):
    """Radians a position of each pair, in 64 bits, and the factor of cosine and sine."""
    dim, base, kind = case["dim"], 10000.0, case["scaling"]
    s, original = SCALINGS[kind].get("scale", 1.0), SCALINGS[kind].get("original", 0)
    i = np.arange(dim // 2, dtype=np.float64)
    if kind == "ntk":
        base *= s ** (dim / (dim - 2.0))
    f = base ** (-2.0 * i / dim)
    if kind == "linear":
        return f / s, 1.0
    if kind == "yarn":  # pairs that turn more than 32 times in the original length are kept, those below once divided
        edge = [dim * math.log(original / (turns * 2.0 * math.pi)) / (2.0 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), dim - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / s * ramp + f * (1.0 - ramp), 0.1 * math.log(s) + 1.0
    if kind == "bands":  # by wavelength: below a quarter of the original length kept, above it divided, between them mixed
        x = np.clip((original * f / (2.0 * math.pi) - 1.0) / 3.0, 0.0, 1.0)
        return f * ((1.0 - x) / s + x), 1.0
    return f, 1.0


def _depths(case, seed):
    """Depths [B, N] of breadth-first draft trees, -1 from a sequence's node count on."""
    B, N = case["B"], case["N"]
    rng = np.random.default_rng([seed, 5])
    parent, depth = np.full((B, N), -1, np.int64), np.zeros((B, N), np.int32)
    rows = np.arange(B)
    for i in range(1, N):
        lo = np.maximum(parent[:, i - 1], (i - 1) // 4)
        parent[:, i] = rng.integers(lo, np.minimum(i, lo + 3))
        depth[:, i] = depth[rows, parent[:, i]] + 1
    return np.where(np.arange(N)[None, :] < _counts(case)[:, None], depth, -1).astype(np.int32)


def prepare(case, seed):
    kind = case["kind"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "logprobs":
        B, P, V, td = case["B"], case["P"], case["V"], DTYPES[case["dtype"]]
        z = torch.empty(B, P, V, dtype=td, device="cuda").normal_(0.0, 2.5, generator=g)
        # tokens as a sampler takes them (the largest of logits and Gumbel noise), none after a step's end
        tokens = torch.empty(B, P, dtype=torch.int32, device="cuda")
        for b in range(B):
            u = torch.rand(P, V, generator=g, device="cuda").clamp_(1e-7, 1.0 - 1e-6)
            tokens[b] = (z[b].float() / case["temperature"] - torch.log(-torch.log(u))).argmax(-1).int()
        asked = torch.from_numpy(_asked(case)).cuda()
        tokens[torch.arange(P, device="cuda")[None, :] >= asked[:, None]] = -1
        return dict(kind=kind, logits=z, tokens=tokens, top=case["top"], temperature=case["temperature"])
    td, lens = DTYPES[case["dtype"]], _lengths(case)
    s = dict(kind=kind, page_size=case["page_size"], cache_len=torch.from_numpy(lens.astype(np.int32)).cuda())
    if kind == "rotary":
        B, N, D = case["B"], case["N"], case["D"]
        n = _counts(case)
        s["n_nodes"] = torch.from_numpy(n.astype(np.int32)).cuda()
        k, v, s["page_table"] = _pool(case, lens + n, g, seed, 1)
        s["k_cache"], s["v_cache"] = k[0], v[0]
        for name, heads in (("q", case["heads"]), ("k", case["kv_heads"]), ("v", case["kv_heads"])):
            s[name] = torch.randn(B, N, heads, D, generator=g, device="cuda").to(td)
        s["positions"] = s["cache_len"] + case["shift"]
        s["depth"] = torch.from_numpy(_depths(case, seed)).cuda() if case["tree"] else None
        s["interleaved"], s["dim"], s["scaling"] = case["interleaved"], case["dim"], case["scaling"]
        f, s["factor"] = _frequencies(case)
        s["frequencies"] = torch.from_numpy(f).cuda()
        return s
    if kind == "weigh":
        B, N, W, H, G, D = (case[x] for x in ("B", "N", "W", "kv_heads", "group", "D"))
        count = _rows(case)
        rng = np.random.default_rng([seed, 9])
        path = np.full((B, W), -1, np.int32)
        for b in range(B):
            path[b, 0] = 0
            path[b, 1:count[b]] = np.sort(rng.choice(np.arange(1, N), size=count[b] - 1, replace=False))
        k, _, s["page_table"] = _pool(case, lens + count, g, seed, 1)
        s["k_cache"] = k[0]
        s["q"] = (1.5 * torch.randn(B, N, H * G, D, generator=g, device="cuda")).to(td)
        s["path"] = None if W == N else torch.from_numpy(path).cuda()
        s["accept"] = None if W == N else torch.from_numpy((count - 1).astype(np.int32)).cuda()
        s["weights"] = torch.rand(B, H, s["page_table"].shape[1] * case["page_size"], generator=g, device="cuda")
        # what the attention's call left: the rows' log-sums
        s["lse"] = torch.zeros(B, N, H * G, device="cuda")
        for b in range(B):
            x, keys, see = _scored(case, s, b, path, torch.float32)
            z = torch.einsum("nhgd,thd->nhgt", x, keys) / math.sqrt(D)
            z = z.masked_fill_(~see[:, None, None, :], -math.inf)
            s["lse"][b, torch.from_numpy(path[b, :count[b]]).long().cuda()] = torch.logsumexp(z, -1).reshape(-1, H * G)
        return s
    layers, B, H = case["layers"], case["B"], case["kv_heads"]
    s["k_cache"], s["v_cache"], s["page_table"] = _pool(case, lens, g, seed, layers)
    T = s["page_table"].shape[1] * case["page_size"]
    # accumulated weights: a few heavy positions, many light ones, some never looked at
    w = torch.empty(layers, B, H, T, device="cuda").normal_(generator=g).mul_(2.0).exp_()
    w *= torch.rand(layers, B, H, T, generator=g, device="cuda") > 0.1
    s["weights"] = w * (torch.arange(T, device="cuda") < s["cache_len"][:, None])[None, :, None, :]
    s["budget"] = torch.full((B,), case["budget"], dtype=torch.int32, device="cuda")
    s["most"], s["sink"], s["recent"] = case["budget"], case["sink"], case["recent"]
    return s


def _scored(case, s, b, path, dtype):
    """Sequence b's weighed rows [n, H, G, D], its keys [T, H, D] and which of them each row sees."""
    H, G, D = case["kv_heads"], case["group"], case["D"]
    L, n = int(_lengths(case)[b]), int(_rows(case)[b])
    pages = s["page_table"][b][:-(-(L + n) // case["page_size"])].long()
    keys = s["k_cache"][pages].flatten(0, 1)[:L + n].to(dtype)
    rows = s["q"][b, torch.from_numpy(path[b, :n]).long().cuda()] if case["W"] != case["N"] else s["q"][b, :n]
    if case["W"] == case["N"]:
        path[b, :n] = np.arange(n)
    see = torch.arange(L + n, device="cuda")[None, :] <= L + torch.arange(n, device="cuda")[:, None]
    return rows.to(dtype).reshape(n, H, G, D), keys, see


def _plain_logprobs(s):
    z, tok, T = s["logits"].float(), s["tokens"].long(), s["temperature"]
    there = tok >= 0
    x = tok.clamp(min=0)
    top = z.amax(-1, keepdim=True)
    y = (z - top) / T
    e = y.exp()
    total = e.sum(-1)
    log_total = total.log()
    zx = z.gather(-1, x[..., None])
    logprob = ((zx - top) / T).squeeze(-1) - log_total
    entropy = log_total - (e * y).sum(-1) / total
    place = torch.arange(z.shape[-1], device=z.device)
    rank = ((z > zx) | ((z == zx) & (place < x[..., None]))).sum(-1)
    zero = torch.zeros_like(logprob)
    out = {"logprob": torch.where(there, logprob, zero), "entropy": torch.where(there, entropy, zero),
           "rank": torch.where(there, rank, torch.full_like(rank, -1)).to(torch.int32)}
    if s["top"]:
        best, at = torch.sort(z, dim=-1, descending=True, stable=True)
        best, at = best[..., :s["top"]], at[..., :s["top"]]
        best = (best - top) / T - log_total[..., None]
        out["top_tokens"] = torch.where(there[..., None], at, torch.full_like(at, -1)).to(torch.int32)
        out["top_logprobs"] = torch.where(there[..., None], best, torch.full_like(best, -math.inf))
    return out


def _turned(x, cos, sin, dim, interleaved):
    """x [.., heads, D] with its first `dim` columns rotated by the angles of cos, sin [.., dim / 2]."""
    if interleaved:
        a, b = x[..., 0:dim:2], x[..., 1:dim:2]
    else:
        a, b = x[..., :dim // 2], x[..., dim // 2:dim]
    cos, sin = cos[..., None, :], sin[..., None, :]
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., dim:]], -1)


def _angles(s):
    B, N = s["q"].shape[:2]
    i = torch.arange(N, device=s["q"].device)[None, :].expand(B, N) if s["depth"] is None else s["depth"].clamp(min=0)
    return (s["positions"].double()[:, None] + i.double())[..., None] * s["frequencies"]


def _slots(s, position):
    """Row of the flattened [pages * page_size] cache that holds each sequence's position."""
    ps = s["page_size"]
    return s["page_table"].long().gather(1, position // ps) * ps + position % ps


def _plain_rotary(s):
    B, N = s["q"].shape[:2]
    angle = _angles(s)
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    i = torch.arange(N, device=s["q"].device)[None, :].expand(B, N)
    used = i < s["n_nodes"].long()[:, None]
    q = _turned(s["q"].float(), cos, sin, s["dim"], s["interleaved"]) * used[:, :, None, None]
    k = _turned(s["k"].float(), cos, sin, s["dim"], s["interleaved"]).to(s["k"].dtype)
    i = torch.where(used, i, torch.zeros_like(i))  # padding repeats node 0
    at = _slots(s, s["cache_len"].long()[:, None] + i)
    pick = i[:, :, None, None].expand(B, N, *k.shape[2:])
    for new, cache in ((k, s["k_cache"]), (s["v"], s["v_cache"])):
        cache.view(-1, *cache.shape[2:])[at] = new.gather(1, pick)
    return {"q": q.to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_weigh(s):
    q, ps, weights = s["q"], s["page_size"], s["weights"]
    B, N, Hq, D = q.shape
    _, H, T = weights.shape
    G = Hq // H
    if s["path"] is None:
        rows, count = torch.arange(N, device=q.device)[None, :].expand(B, N), torch.full((B,), N, device=q.device)
    else:
        rows, count = s["path"].long().clamp(min=0), s["accept"].long() + 1
    W = rows.shape[1]
    x = q.gather(1, rows[:, :, None, None].expand(B, W, Hq, D)).float()
    lse = s["lse"].gather(1, rows[:, :, None].expand(B, W, Hq))
    keys = s["k_cache"][s["page_table"].long().clamp(min=0)].reshape(B, T, H, D).float()
    x = x.reshape(B, W, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, W * G, D)
    score = ((x @ keys.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))).reshape(B, H, W, G, T)
    row = torch.arange(W, device=q.device)
    seen = torch.arange(T, device=q.device)[None, None, :] <= (s["cache_len"].long()[:, None] + row)[:, :, None]
    seen = seen & (row[None, :] < count[:, None])[:, :, None]
    score -= lse.reshape(B, W, H, G).permute(0, 2, 1, 3)[..., None]
    p = score.masked_fill_(~seen[:, None, :, None, :], -math.inf).exp_()
    weights += p.sum((2, 3))
    return {"weights": weights}


def _plain_evict(s):
    k, v, ps, lens = s["k_cache"], s["v_cache"], s["page_size"], s["cache_len"].long()
    w = s["weights"].clone()  # (a program evicts on; a pass here begins with the same weights)
    Y, B, H, T = w.shape
    D, K = k.shape[-1], s["most"]
    place = torch.arange(T, device=w.device)[None, :]
    new_len = torch.minimum(lens, s["budget"].long())
    over = (lens > new_len)[:, None]
    # sinks and recent positions first, then the rest by weight (ties: the lowest position), then what is not there
    always = (place < s["sink"]) | (place >= lens[:, None] - s["recent"]) | ~over
    order = torch.where(always[None, :, None, :], torch.full_like(w, math.inf), w)
    order = order.masked_fill_((place >= lens[:, None])[None, :, None, :], -math.inf)
    best = torch.sort(order, dim=-1, descending=True, stable=True).indices[..., :K]
    i = torch.arange(best.shape[-1], device=w.device)
    there = (i < new_len[:, None])[None, :, None, :]
    source = torch.where(there, best, torch.full_like(best, T)).sort(-1).values  # ascending, T where there is none
    stay = ~over[None, :, None, :] | (source >= T)
    # what stays goes onto itself; what is past the end repeats position 0 (an empty sequence has no pages: page 0's slot 0)
    target = torch.where(source >= T, torch.zeros_like(source), i.expand_as(source))
    source = torch.where(stay, target, source)
    page = s["page_table"].long().clamp(min=0)[None, :, None, :].expand(Y, B, H, -1)
    to = page.gather(-1, target // ps) * ps + target % ps
    frm = page.gather(-1, source // ps) * ps + source % ps
    layer = torch.arange(Y, device=w.device)[:, None, None, None]
    head = torch.arange(H, device=w.device)[None, None, :, None]
    first = target == 0
    keep = ~first | (i == 0)  # (only the true position 0 is written)
    for cache in (k, v):
        flat = cache.view(Y, -1, H, D)
        moved = flat[layer, frm, head]
        where = (keep & there).nonzero(as_tuple=True)
        flat[where[0], to[where], where[2]] = moved[where]
    kept = w.gather(-1, source)
    w[..., :kept.shape[-1]] = torch.where(there, kept, w[..., :kept.shape[-1]])
    w.masked_fill_(((place >= new_len[:, None]) & (place < lens[:, None]))[None, :, None, :], 0.0)
    return {"k_cache": k, "v_cache": v, "weights": w, "cache_len": new_len.to(torch.int32)}


def _own(s):
    import speculative_decoding_verification_05_gb300 as sv

    kind = s["kind"]
    if kind == "logprobs":
        r = sv.token_logprobs(s["logits"], s["tokens"], top=s["top"], temperature=s["temperature"])
        names = ("logprob", "entropy", "rank") + (("top_tokens", "top_logprobs") if s["top"] else ())
        return {n: r[n] for n in names}
    if kind == "rotary":
        if "plan" not in s:  # made once, kept with the model
            s["plan"] = sv.rotary(s["dim"], base=10000.0, interleaved=s["interleaved"], **SCALINGS[s["scaling"]])
        r = sv.cache_append_rotary(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["cache_len"],
                                   s["plan"], positions=s["positions"], depth=s["depth"], n_nodes=s["n_nodes"])
        return {"q": r["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if kind == "weigh":
        sv.cache_weigh(s["q"], s["lse"], s["k_cache"], s["page_table"], s["cache_len"], s["weights"],
                       accept_len=s["accept"], path_nodes=s["path"])
        return {"weights": s["weights"]}
    w = s["weights"].clone()
    r = sv.cache_evict(s["k_cache"], s["v_cache"], s["page_table"], s["cache_len"], w, s["budget"], sink=s["sink"],
                       recent=s["recent"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": w, "cache_len": r["cache_len"]}


def run(state):
    if own:
        return _own(state)
    return {"logprobs": _plain_logprobs, "rotary": _plain_rotary, "weigh": _plain_weigh,
            "evict": _plain_evict}[state["kind"]](state)


def work(case):
    es, kind = ESIZE[case["dtype"]], case["kind"]
    if kind == "logprobs":
        rows = float(_asked(case).sum())
        return {"bytes": rows * case["V"] * es + case["B"] * case["P"] * (16.0 + 8.0 * case["top"]),
                "flops": 6.0 * rows * case["V"]}
    lens, H, D = _lengths(case), case["kv_heads"], case["D"]
    if kind == "rotary":
        n = float(_counts(case).sum())
        return {"bytes": n * (2.0 * case["heads"] + 4.0 * H) * D * es, "flops": 3.0 * n * (case["heads"] + H) * case["dim"]}
    if kind == "weigh":
        n, G = _rows(case), case["group"]
        keys = float((lens + n).sum()) * H
        return {"bytes": keys * (D * es + 8.0) + float(n.sum()) * H * G * (D * es + 4.0),
                "flops": 2.0 * D * float((n * lens + n * (n + 1) / 2.0).sum()) * H * G}
    over = float(case["B"] if case["B"] == 1 and lens[0] > case["budget"] else (lens > case["budget"]).sum())
    seen = float(lens[lens > case["budget"]].sum())
    rows = over * case["layers"] * H
    # kept keys and values read and written (the sinks stay), weights read and written
    return {"bytes": max(64.0 * case["B"], rows * (case["budget"] - case["sink"]) * 4.0 * D * es
                         + 8.0 * seen * case["layers"] * H), "flops": 0.0}


def exact(case, seed):
    """From the definitions, one sequence at a time, in 64 bits; what an eviction returns is chosen and moved, not
    computed."""
    kind = case["kind"]
    if kind == "evict":
        return None
    s = prepare(case, seed)
    if kind == "logprobs":
        B, P, top = case["B"], case["P"], case["top"]
        f64 = dict(dtype=torch.float64, device="cuda")
        out = {"logprob": torch.zeros(B, P, **f64), "entropy": torch.zeros(B, P, **f64), "rank": None}
        if top:
            out["top_tokens"], out["top_logprobs"] = None, torch.full((B, P, top), -math.inf, **f64)
        for b in range(B):
            n = int(_asked(case)[b])
            for at in range(0, n, 64):
                rows = slice(at, min(n, at + 64))
                lp = torch.log_softmax(s["logits"][b, rows].double() / case["temperature"], dim=-1)
                out["logprob"][b, rows] = lp.gather(-1, s["tokens"][b, rows].long()[:, None])[:, 0]
                out["entropy"][b, rows] = -(lp.exp() * lp).sum(-1)
                if top:
                    out["top_logprobs"][b, rows] = lp.topk(top, dim=-1).values
        return out
    if kind == "rotary":
        D, dim, n = case["D"], case["dim"], _counts(case)
        f, factor = _frequencies(case)
        keys, q = s["k_cache"].double(), torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        pair = torch.arange(dim // 2, device="cuda")
        first = 2 * pair if case["interleaved"] else pair
        second = first + (1 if case["interleaved"] else dim // 2)
        for b in range(case["B"]):
            steps = torch.arange(n[b], device="cuda") if s["depth"] is None else s["depth"][b, :n[b]]
            angle = torch.outer((int(s["positions"][b]) + steps).double(), torch.from_numpy(f).cuda())
            turn = torch.polar(torch.full_like(angle, factor), angle)[:, None, :]
            t = torch.arange(n[b], device="cuda") + int(s["cache_len"][b])
            page, slot = s["page_table"][b].long()[t // case["page_size"]], t % case["page_size"]
            for name, put in (("q", None), ("k", (page, slot))):
                x = s[name][b, :n[b]].double()
                y = torch.complex(x[..., first], x[..., second]) * turn
                x[..., first], x[..., second] = y.real, y.imag
                if put is None:
                    q[b, :n[b]] = x
                else:
                    keys[put] = x
        return {"q": q, "k_cache": keys, "v_cache": None}
    H, G, D = case["kv_heads"], case["group"], case["D"]
    weights = s["weights"].double()
    path = np.zeros((case["B"], case["W"]), np.int32) if s["path"] is None else s["path"].cpu().numpy()
    for b in range(case["B"]):
        x, keys, see = _scored(case, s, b, path, torch.float64)
        lse = s["lse"][b, torch.from_numpy(path[b, :len(x)]).long().cuda()].double().reshape(-1, H, G)
        for h in range(H):
            z = torch.einsum("ngd,td->gnt", x[:, h], keys[:, h]) / math.sqrt(D)
            p = torch.where(see, (z - lse[:, h].T[..., None]).exp(), torch.zeros_like(z))
            weights[b, h, :len(keys)] += p.sum((0, 1))
    return {"weights": weights}
