"""One decoder layer that checks trees of drafted tokens, weights and cache quantized.

The projections are packed mxfp8 weights (nvfp4_mx_mm_packed), the experts NVFP4
weights, keys and values a paged NVFP4 cache.  A step takes a few sequences'
drafted tokens, all in one batch:

    n, r = norm(x + r)               nvfp4_mx_rms_norm, in the product's layout
    qkv = n W_qkv^T                  one product; q, k and v are slices of it
    q, cache[slots] <- k, v          nvfp4_kv_write_rotated
    a = attention(q, cache, tree)    nvfp4_kv_tree_attention
    n, r = norm(a W_out^T + r)       nvfp4_mx_rms_norm, in x's type
    x' = experts(n)                  nvfp4_moe

After a step one path of each tree is accepted: its tokens stay, and the next
step writes over the rest, its tree a chain of the accepted tokens with new
drafts behind them.

    python examples/draft_tree_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_amd as nv  # noqa: E402

HIDDEN, QUERY_HEADS, HEADS, DIM = 512, 8, 2, 64
EXPERTS, TOP_K, INNER = 8, 2, 384
PAGE, LONGEST = 16, 512


class Layer:
    """The weights, quantized once, and the cache that the layer fills."""

    def __init__(self, pages, seed=0):
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, size=1.0):
            return (torch.randn(*shape, generator=gen) * size).to(torch.bfloat16).cuda()

        def packed(n, k):
            return nv.nvfp4_mx_pack(*nv.nvfp4_mx_quantize(normal(n, k, size=k ** -0.5), "mxfp8"), "mxfp8")

        def experts(n, k):
            w = [normal(n, k, size=k ** -0.5) for _ in range(EXPERTS)]
            g = [nv.nvfp4_tensor_amax(x) for x in w]
            codes, scales = zip(*(nv.nvfp4_quantize(x, y) for x, y in zip(w, g)))
            return torch.stack(codes), torch.stack(scales), torch.cat(g)

        self.norms = [1 + normal(HIDDEN, size=0.1) for _ in range(2)]
        self.qkv = packed((QUERY_HEADS + 2 * HEADS) * DIM, HIDDEN)
        self.out = packed(HIDDEN, QUERY_HEADS * DIM)
        self.router = normal(EXPERTS, HIDDEN, size=HIDDEN ** -0.5)
        self.gate_up, self.down = experts(2 * INNER, HIDDEN), experts(HIDDEN, INNER)
        self.table = nv.rotation_table(LONGEST, DIM)
        # fixed global scales: an upper bound of the keys' and values' magnitudes
        bound = torch.tensor([16.0], device="cuda")
        self.cache = nv.kv_cache(pages, PAGE, HEADS, DIM, global_scale_k=bound, global_scale_v=bound)

    def __call__(self, x, residual, slots, positions, pages, lens, starts, tree, max_queries, max_context):
        """x, residual [tokens, HIDDEN] -> all that the step computes, by name."""
        n1 = nv.nvfp4_mx_rms_norm(x, self.norms[0], "mxfp8", residual, packed=True)
        qkv = nv.nvfp4_mx_mm_packed(n1.quantized, self.qkv).view(len(x), -1, DIM)
        q, k, v = qkv.split([QUERY_HEADS, HEADS, HEADS], 1)  # no copies
        rotated = nv.nvfp4_kv_write_rotated(self.cache, k, v, slots, positions, self.table, q=q)
        a, lse = nv.nvfp4_kv_tree_attention(rotated, self.cache, pages, lens, starts, tree, max_queries=max_queries,
                                            max_context=max_context, return_lse=True)
        y = nv.nvfp4_mx_mm_packed(nv.nvfp4_mx_quantize_packed(a.view(len(x), -1), "mxfp8"), self.out)
        n2 = nv.nvfp4_mx_rms_norm(y, self.norms[1], "mxfp8", n1.sum, normed=True)
        out, chosen, weights = nv.nvfp4_moe(n2.normed, *self.gate_up[:2], *self.down[:2], router=self.router, top_k=TOP_K,
                                            global_scale_gate_up=self.gate_up[2], global_scale_down=self.down[2])
        return dict(n1=n1, qkv=qkv, rotated=rotated, attention=a, lse=lse, projected=y, n2=n2, chosen=chosen, weights=weights,
                    out=out)


def batch(layer_pages, settled, parents):
    """What a step needs besides its tokens: `settled` tokens of each sequence are in the cache, its drafts hang
    together as `parents` says."""
    counts = [len(p) for p in parents]
    tree, depths = nv.kv_trees(parents)
    base = torch.repeat_interleave(torch.tensor(settled), torch.tensor(counts))
    place = base + torch.cat([torch.arange(n) for n in counts])
    rows = torch.repeat_interleave(layer_pages, torch.tensor(counts), 0)
    slots = rows.gather(1, (place // PAGE)[:, None]).view(-1).long() * PAGE + place % PAGE
    lens = [s + n for s, n in zip(settled, counts)]
    starts = torch.tensor([0, *counts]).cumsum(0)
    whole = dict(slots=slots, positions=(base + depths).int(), pages=layer_pages, lens=torch.tensor(lens, dtype=torch.int32),
                 starts=starts.int(), tree=tree)
    return {**{n: t.cuda() for n, t in whole.items()}, "max_queries": max(counts), "max_context": max(lens)}


def draft(gen, chain, n):
    """A tree of `n` drafts behind a chain of `chain` accepted tokens."""
    return [d - 1 for d in range(chain)] + [chain - 1 + int(torch.randint(0, d + 1, (1,), generator=gen)) for d in range(n)]


def path(parents):
    """The deepest draft and its ancestors, first to last."""
    depth = []
    for p in parents:
        depth.append(depth[p] + 1 if p >= 0 else 0)
    at, found = depth.index(max(depth)), []
    while at >= 0:
        found.insert(0, at)
        at = parents[at]
    return found


def run(prompts=(13, 1, 20), drafts=6, steps=3, seed=1):
    """Serves the prompts, as chains, and `steps` trees of `drafts` tokens each; returns the tokens in the cache in
    the end and the last step's hidden states."""
    gen = torch.Generator().manual_seed(seed)
    seqs = len(prompts)
    per_seq = -(-(max(prompts) + steps * (drafts + 2)) // PAGE) + 1
    # pages in no particular order, as an allocator hands them out
    pages = torch.randperm(seqs * per_seq, generator=gen).to(torch.int32).view(seqs, per_seq)
    layer = Layer(seqs * per_seq)

    def hidden(n):
        return torch.randn(n, HIDDEN, generator=gen).to(torch.bfloat16).cuda()

    settled, parents = [0] * seqs, [draft(gen, n, 0) for n in prompts]
    tokens = [hidden(n) for n in prompts]
    for step in range(steps + 1):
        x = torch.cat(tokens)
        got = layer(x, torch.zeros_like(x), **batch(pages, settled, parents))
        if step == steps:
            break
        ends = [0]
        for p in parents:
            ends.append(ends[-1] + len(p))
        for b in range(seqs):
            kept = path(parents[b])
            here = tokens[b][kept]
            # what the accepted path holds as a prefix of the batch is settled, the rest comes again as a chain
            whole = sum(1 for i, d in enumerate(kept) if i == d)
            settled[b] += whole
            # (one token at least comes again: the drafts hang on it)
            back = here[whole:] if whole < len(kept) else hidden(1)
            parents[b] = draft(gen, len(back), drafts)
            tokens[b] = torch.cat([back, hidden(drafts)])
    return [s + len(p) for s, p in zip(settled, parents)], got["out"]


if __name__ == "__main__":
    lengths, out = run()
    print("tokens in the cache:", lengths, "  hidden states:", tuple(out.shape), "finite:", bool(torch.isfinite(out).all()))
