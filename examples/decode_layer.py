"""One attention layer served with weights and cache in NVFP4.

The layer's projections are packed NVFP4 weights (nvfp4_qqmm_packed); its keys
and values go into a paged NVFP4 cache.  A few sequences of different lengths
are taken in as one batch of prompts, then continued token by token:

    qkv = x W_qkv^T                 one product; q, k and v are slices of it
    cache[slots] <- k, v            nvfp4_kv_write
    a = attention(q, cache)         nvfp4_kv_attention
    x' = a W_out^T

and at the end the same layer is computed once more from what the cache holds
(nvfp4_kv_read), in float32 with torch, to show what the cache returns.

    python examples/decode_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_amd as nv  # noqa: E402

HIDDEN, QUERY_HEADS, HEADS, DIM = 1024, 16, 4, 64
PAGE = 16


class Layer:
    """The projections, quantized and packed once, and the cache they fill."""

    def __init__(self, pages, seed=0):
        gen = torch.Generator().manual_seed(seed)

        def weight(n, k):
            w = (torch.randn(n, k, generator=gen) * k ** -0.5).to(torch.bfloat16).cuda()
            g = nv.nvfp4_tensor_amax(w)
            return nv.nvfp4_mfma_pack(*nv.nvfp4_quantize(w, g)), g

        self.qkv, self.g_qkv = weight((QUERY_HEADS + 2 * HEADS) * DIM, HIDDEN)
        self.out, self.g_out = weight(HIDDEN, QUERY_HEADS * DIM)
        # fixed global scales: an upper bound of the keys' and values' magnitudes
        bound = torch.tensor([16.0], device="cuda")
        self.cache = nv.kv_cache(pages, PAGE, HEADS, DIM, global_scale_k=bound, global_scale_v=bound)

    def __call__(self, x, slots, table, context_lens, query_starts=None, max_queries=1, max_context=None):
        """x [tokens, HIDDEN] -> (the layer's output, q, the attention's output)."""
        qkv = nv.nvfp4_qqmm_packed(x, self.qkv, nv.nvfp4_tensor_amax(x), self.g_qkv)
        q, k, v = qkv.view(len(x), -1, DIM).split([QUERY_HEADS, HEADS, HEADS], 1)  # no copies
        nv.nvfp4_kv_write(self.cache, k, v, slots)
        a = nv.nvfp4_kv_attention(q, self.cache, table, context_lens, query_starts, max_queries, max_context)
        flat = a.reshape(len(x), -1)
        return nv.nvfp4_qqmm_packed(flat, self.out, nv.nvfp4_tensor_amax(flat), self.g_out), q, a


def slots_of(table, b, positions):
    """Slots of `positions` of sequence b."""
    return table[b, positions // PAGE].long() * PAGE + positions % PAGE


def run(prompts=(37, 5, 64, 1), steps=8, seed=1):
    """Serves the prompts and `steps` more tokens of each; returns the largest difference of the last
    step's attention from torch's over the cache read back, relative to its largest value."""
    seqs, longest = len(prompts), max(prompts) + steps
    per_seq = -(-longest // PAGE)
    gen = torch.Generator().manual_seed(seed)
    # pages in no particular order, as an allocator hands them out
    table = torch.randperm(seqs * per_seq, generator=gen).to(torch.int32).view(seqs, per_seq)
    layer = Layer(seqs * per_seq)

    # the prompts, one behind the other in a batch
    starts = torch.tensor([0, *prompts]).cumsum(0).to(torch.int32)
    slots = torch.cat([slots_of(table, b, torch.arange(n)) for b, n in enumerate(prompts)]).cuda()
    x = torch.randn(sum(prompts), HIDDEN, generator=gen).to(torch.bfloat16).cuda()
    lens = torch.tensor(prompts, dtype=torch.int32)
    dev_table = table.cuda()
    y, _, _ = layer(x, slots, dev_table, lens.cuda(), starts.cuda(), max(prompts), max(prompts))
    x = y[(starts[1:] - 1).long().cuda()].contiguous()  # the last token of each

    for _ in range(steps):
        slots = torch.stack([slots_of(table, b, lens[b]) for b in range(seqs)]).cuda()
        lens = lens + 1
        x, q, a = layer(x, slots, dev_table, lens.cuda(), max_context=longest)

    # the last step's attention from the cache's contents
    worst = 0.0
    for b in range(seqs):
        k, v = nv.nvfp4_kv_read(layer.cache, slots_of(table, b, torch.arange(int(lens[b]))).cuda(), torch.float32)
        k, v = (t.repeat_interleave(QUERY_HEADS // HEADS, 1).permute(1, 0, 2) for t in (k, v))  # [heads, keys, dim]
        s = (k * q[b].float()[:, None]).sum(-1) * DIM ** -0.5
        ref = (s.softmax(-1)[..., None] * v).sum(1)
        worst = max(worst, float((a[b].float() - ref).abs().max() / ref.abs().max()))
    return worst


if __name__ == "__main__":
    print(f"largest difference from the cache read back: {run():.2e} of the largest value (bfloat16: 3.9e-03)")
