"""Tree-speculative decoding of a small random model over a paged cache.

One prompt is read once and shared by several branches (``cache_fork``); every
step then takes pages for a draft tree (``cache_resize``), builds it
(``tree_build``), writes its keys and values (``cache_append``), lets its nodes
attend to the context and their ancestors (``tree_attention``), verifies it
(``verify_tree``) and keeps the accepted path's entries (``cache_compact``).
The drafts are the model's own continuations with some tokens replaced. With
greedy verification the result is that of decoding token by token, which the
example checks.

    python examples/paged_tree_decode.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_05_gb300 as sv  # noqa: E402


class Model:
    """A decoder with random weights: attention and a gated layer, no training."""

    def __init__(self, vocab=211, layers=2, kv_heads=2, group=4, D=64, dtype=torch.float32, seed=0):
        g = torch.Generator().manual_seed(seed)
        w = lambda *shape: (torch.randn(*shape, generator=g) * shape[0] ** -0.5).to(dtype).cuda()
        self.V, self.layers, self.Hkv, self.H, self.D, self.dtype = vocab, layers, kv_heads, kv_heads * group, D, dtype
        self.hidden = self.H * D
        self.embed = w(vocab, self.hidden) * vocab ** 0.5
        self.qkv = [w(self.hidden, (self.H + 2 * kv_heads) * D) for _ in range(layers)]
        self.proj = [w(self.hidden, self.hidden) for _ in range(layers)]
        self.gate = [w(self.hidden, 2 * self.hidden) for _ in range(layers)]
        self.head = w(self.hidden, vocab)
        self.freq = 1000.0 ** (-torch.arange(self.hidden // 2, device="cuda") / (self.hidden // 2))

    def norm(self, x):
        return torch.nn.functional.layer_norm(x.float(), (self.hidden,)).to(self.dtype)

    def forward(self, tokens, depth, cache, table, cache_len, mask=None, n_nodes=None):
        """Logits [B, N, V] of the nodes, whose keys and values go to the cache."""
        B, N = tokens.shape
        at = (cache_len[:, None] + depth).float()[..., None] * self.freq
        x = self.embed[tokens.long()] + torch.cat([at.sin(), at.cos()], -1).to(self.dtype)
        for l in range(self.layers):
            q, k, v = (self.norm(x) @ self.qkv[l]).view(B, N, -1, self.D).split([self.H, self.Hkv, self.Hkv], 2)
            sv.cache_append(k, v, cache.k[l], cache.v[l], table, cache_len, n_nodes, cache.refs)
            a = sv.tree_attention(q, cache.k[l], cache.v[l], table, cache_len, mask, n_nodes)["out"]
            x = x + a.reshape(B, N, -1) @ self.proj[l]
            u, g = (self.norm(x) @ self.gate[l]).chunk(2, -1)
            x = x + u * torch.sigmoid(g)
        return (self.norm(x) @ self.head).float()


class Cache:
    """Pages of every layer, the sequences' page table and lengths."""

    def __init__(self, model, seqs, max_tokens, page_size=16):
        self.ps, width = page_size, -(-max_tokens // page_size)
        pages = seqs * width
        self.k, self.v = (torch.zeros(model.layers, pages, page_size, model.Hkv, model.D, dtype=model.dtype,
                                      device="cuda") for _ in range(2))
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table, self.refs = torch.full((seqs, width), -1, **i32), torch.zeros(pages, **i32)
        self.len = torch.zeros(seqs, **i32)

    def resize(self, seqs, tokens):
        status = sv.cache_resize(self.table, self.refs, seqs, tokens, self.ps)["status"]
        if status.any():
            raise RuntimeError(f"no pages: {status.tolist()}")


def start(model, prompt, branches, max_tokens):
    """The prompt in sequence 0 and its branches 1 .. branches; the prompt's last logits."""
    c = Cache(model, branches + 1, max_tokens)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = len(prompt)
    c.resize(one, one + n)
    tokens = torch.tensor([prompt], dtype=torch.int32, device="cuda")
    z = model.forward(tokens, torch.arange(n, device="cuda"), c, c.table[:1], c.len[:1])[0, -1]
    c.len[0] = n
    dst = torch.arange(1, branches + 1, dtype=torch.int32, device="cuda")
    if sv.cache_fork(c.k, c.v, c.table, c.len, c.refs, torch.zeros_like(dst), dst)["status"].any():
        raise RuntimeError("no pages for the branches")
    return c, dst, z


def plain(model, prompt, branches, steps):
    """Token by token: [branches, steps + 1], branch b's first token the b-th likeliest."""
    c, seqs, z = start(model, prompt, branches, len(prompt) + steps + 1)
    out = [z.topk(branches).indices.int()[:, None]]
    table = c.table[1:]
    for _ in range(steps):
        c.resize(seqs, c.len[1:] + 1)
        z = model.forward(out[-1], torch.zeros(1, device="cuda"), c, table, c.len[1:])
        out.append(z.argmax(-1).int())
        c.len[1:] += 1
    return torch.cat(out, 1)


def speculative(model, prompt, branches, steps, drafts, nodes=12):
    """The same tokens by draft trees; drafts(b, position) gives continuations [C, L]. Returns them and the steps taken."""
    c, seqs, z = start(model, prompt, branches, len(prompt) + steps + nodes + 8)
    root = z.topk(branches).indices.int()
    out, table, calls = [[t] for t in root.tolist()], c.table[1:], 0
    while min(map(len, out)) <= steps:
        cand = torch.stack([drafts(b, min(len(out[b]), steps)) for b in range(branches)]).int().cuda()
        t = sv.tree_build(cand, root, model.V, nodes)
        unused = torch.arange(nodes, device="cuda") >= t["n_nodes"][:, None]
        c.resize(seqs, c.len[1:] + nodes)
        z = model.forward(t["node_tokens"].clamp(min=0), t["depth"].clamp(min=0), c, table, c.len[1:], t["mask"],
                          t["n_nodes"])
        # (places that the tree left unused repeat node 1, which comes before them where it is accepted)
        tok, par, dep = (torch.where(unused, t[k][:, 1:2], t[k]) for k in ("node_tokens", "parent", "depth"))
        r = sv.verify_tree(z, tok, par, dep, cand.shape[2])
        kept = sv.cache_compact(c.k, c.v, table, c.len[1:], r["accept_len"], r["path_nodes"], c.refs)
        if r["status"].any() or kept["status"].any():
            raise RuntimeError((r["status"].tolist(), kept["status"].tolist()))
        c.len[1:] = kept["cache_len"]
        root = r["bonus"]
        for b, (n, row) in enumerate(zip(r["accept_len"].tolist(), r["tokens"].tolist())):
            out[b] += row[:n + 1]
        calls += 1
    return torch.tensor([o[:steps + 1] for o in out], dtype=torch.int32), calls


def run(branches=3, steps=40, prompt_tokens=37, wrong=0.25, dtype=torch.float32, seed=0):
    """Both ways: tokens by plain decoding, by draft trees, and the trees' steps."""
    model = Model(dtype=dtype, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    prompt = torch.randint(model.V, (prompt_tokens,), generator=g).tolist()
    want = plain(model, prompt, branches, steps).cpu()

    def drafts(b, at, count=4, length=5):
        ahead = want[b, at:at + length]
        d = torch.full((count, length), -1, dtype=torch.int32)
        d[:, :len(ahead)] = ahead
        swap = (torch.rand(count, length, generator=g) < wrong) & (d >= 0)
        return torch.where(swap, torch.randint(model.V, d.shape, generator=g, dtype=torch.int32), d)

    got, calls = speculative(model, prompt, branches, steps, drafts)
    return want, got, calls


if __name__ == "__main__":
    want, got, calls = run()
    print("branches", want.shape[0], "tokens each", want.shape[1], "tree steps", calls,
          "same as token by token:", bool((want == got).all()))
