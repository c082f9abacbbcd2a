"""Helpers of the key/value cache tests: caches with stated contents, and the
attention over them in 64 bits on the CPU with an error bound for each output.

The bound (derived from the arithmetic, not from runs).  u is the unit
roundoff of the output type, w = exp(s - lse) the softmax weights, N the keys
seen.  A score's absolute error is at most
    e = (dim + 8) 2^-24 S + c S,   S = max_j scale sum_d |q_d k_jd|
(dim float32 additions of exact products, a multiplication by the scale and
the global factor; c = 2^-22 for float32 queries, which are used as a pair of
float16).  A weight then has the relative error 2 e + 2^-20 (exponential,
running maximum) + p, p = 2^-11 for its rounding to float16 (2^-22 as a pair);
sums over the keys add N 2^-24 each.  So
    |out - ref| <= u |ref| + (p + 4 e + 2^-18 + 2 N 2^-24) sum_j w_j |v_j| (1 + 2 u)
    |lse - ref| <= e + 2^-20 + N 2^-24 + 2^-22 |ref|
plus one subnormal step of the output type.
"""
import torch

import nvfp4_block_scaled_amd as nv

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def e4m3_table():
    t = [(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)]
    t[127] = float("nan")
    return torch.tensor(t + [-v for v in t], dtype=torch.float64)


def e2m1_table():
    t = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(t + [-v for v in t], dtype=torch.float64)


def values(codes, scales, g):
    """float64 values [..., dim] held by codes and scales (CPU uint8) under the global scale g."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    by = e4m3_table()[scales.long()].repeat_interleave(16, -1)
    return e2m1_table()[both] * by * (1.0 if g is None else float(g) / 2688.0)


def random_cache(pages, page_size, heads, dim, seed, g_k=20.0, g_v=6.0, unwritten=()):
    """A cache of random codes and ordinary scales on the GPU; every byte of
    the `unwritten` pages is 255 (scales that are no number)."""
    gen = torch.Generator().manual_seed(seed)
    c = {}
    for n in "kv":
        codes = torch.randint(0, 256, (pages, heads, page_size, dim // 2), dtype=torch.uint8, generator=gen)
        scales = torch.randint(0x38, 0x58, (pages, heads, page_size, dim // 16), dtype=torch.uint8, generator=gen)
        for p in unwritten:
            codes[p], scales[p] = 255, 255
        c[n + "_codes"], c[n + "_scales"] = codes.cuda(), scales.cuda()

    def scalar(g):
        return None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")

    return nv.KVCache(**c, global_scale_k=scalar(g_k), global_scale_v=scalar(g_v))


def reference(q, cache, page_table, context_lens, starts, scale, causal=True, window=0):
    """(out, lse, bound of out, bound of lse) in float64 on the CPU; rows outside every sequence are nan."""
    c = {n: getattr(cache, n).cpu() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    g_k = None if cache.global_scale_k is None else cache.global_scale_k.item()
    g_v = None if cache.global_scale_v is None else cache.global_scale_v.item()
    dtype, u = q.dtype, UNIT[q.dtype]
    p_round = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -11
    x = q.detach().cpu().double()
    tokens, hq, dim = x.shape
    groups = hq // cache.heads
    table, lens = page_table.cpu().tolist(), context_lens.cpu().tolist()
    out = torch.full((tokens, hq, dim), float("nan"), dtype=torch.float64)
    lse = torch.full((tokens, hq), float("nan"), dtype=torch.float64)
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    for b, context in enumerate(lens):
        first, last = starts[b], starts[b + 1]
        n = last - first
        j = [i for i in range(max(context, 0)) if 0 <= table[b][i // cache.page_size] < cache.pages]
        pages = torch.tensor([table[b][i // cache.page_size] for i in j], dtype=torch.long)
        offs = torch.tensor([i % cache.page_size for i in j], dtype=torch.long)
        key = torch.tensor(j, dtype=torch.long)
        for h in range(cache.heads if n else 0):
            k = values(c["k_codes"][pages, h, offs], c["k_scales"][pages, h, offs], g_k)
            v = values(c["v_codes"][pages, h, offs], c["v_scales"][pages, h, offs], g_v)
            for i in range(first, last):
                pos = context - n + (i - first)
                see = (key <= pos) if causal else torch.ones_like(key, dtype=torch.bool)
                if causal and window:
                    see &= key > pos - window
                for a in range(h * groups, (h + 1) * groups):
                    if not see.any():
                        out[i, a], lse[i, a] = 0.0, float("-inf")
                        continue
                    ks, vs = k[see], v[see]
                    s = ks @ x[i, a] * scale
                    lse[i, a] = torch.logsumexp(s, 0)
                    w = torch.exp(s - lse[i, a])
                    out[i, a] = w @ vs
                    size = (ks.abs() @ x[i, a].abs() * scale).max().item()
                    e = (dim + 8) * 2.0 ** -24 * size + (2.0 ** -22 * size if dtype == torch.float32 else 0.0)
                    more = len(s) * 2.0 ** -24
                    bound[i, a] = u * out[i, a].abs() + TINY[dtype] + \
                        (p_round + 4 * e + 2.0 ** -18 + 2 * more) * (w @ vs.abs()) * (1 + 2 * u)
                    lse_bound[i, a] = e + 2.0 ** -20 + more + 2.0 ** -22 * abs(lse[i, a].item())
    return out, lse, bound, lse_bound


def check(got, got_lse, ref, what=""):
    """got against reference()'s answer; rows of no sequence must have kept their nan."""
    out, lse, bound, lse_bound = ref
    got = got.detach().cpu().double()
    outside = torch.isnan(out)
    assert torch.isnan(got[outside]).all(), f"{what}: rows of no sequence were written"
    inside = ~outside
    assert torch.isfinite(got[inside]).all(), f"{what}: not finite"
    off = ((got - out).abs() / bound.clamp(min=1e-300))[inside & (bound > 0)]
    zero = inside & (bound == 0)
    assert (got[zero] == 0).all(), f"{what}: a row that sees nothing is not zero"
    worst = off.max().item() if off.numel() else 0.0
    print(f"  {what}: worst error / bound = {worst:.3f}", flush=True)
    assert worst <= 1.0, (what, worst)
    if got_lse is not None:
        got_lse = got_lse.detach().cpu().double()
        none = torch.isinf(lse)
        assert (got_lse[none] == float("-inf")).all(), f"{what}: lse of a row that sees nothing"
        fine = torch.isfinite(lse)
        assert ((got_lse - lse).abs()[fine] <= lse_bound[fine]).all(), \
            (what, ((got_lse - lse).abs() / lse_bound)[fine].max().item())
