"""Measured cases of the NVFP4 key/value cache: writing it, reading it back, and attention over it.

A cache holds `pages` pages of `page` tokens.  For every token and kv head it keeps the head's `dim` values as
e2m1 codes (two to a byte, element 2j in the low nibble) and one e4m3 scale per 16 values; a value is
e2m1(code) * e4m3(scale) * g / 2688 with a float32 global scale g each for keys and values.

Four kinds of case:
  write   quantise the keys and values of new tokens into their slots, and return what those slots then hold
  read    return the keys and values of given slots
  single  attention of one query token (or a few) per sequence over its cached context
  prompt  causal attention of the last `queries` tokens of each sequence over its cached context

`own` false: elementary torch operations in 32 bits.  `own` true: the package's calls on the same inputs.
"""
import math

import torch

own = False

GROUP = 16
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One decoding step of 64 sequences: each appends one token; the latency of a small call counts.
        dict(name="write 64 single tokens", kind="write", tokens=64, heads=8, dim=128, page=16, dtype="bf16",
             fused=True, padded=0),
        # A batch of prompts, keys and values as slices of the fused projection's output.
        dict(name="write 16384 prompt tokens", kind="write", tokens=16384, heads=8, dim=128, page=64, dtype="bf16",
             fused=True, padded=0),
        # Odd sizes: heads of 80 values, a page that is no power of two, some tokens of the batch padding.
        dict(name="write 3001 tokens, dim 80", kind="write", tokens=3001, heads=5, dim=80, page=24, dtype="f16",
             fused=False, padded=13),
        # A long shared prefix brought back to 16 bits (to move it, or for a path that wants it whole).
        dict(name="read 65536 tokens", kind="read", tokens=65536, heads=8, dim=128, page=64, dtype="bf16", padded=0),
        # A short one in float32, odd in every size.
        dict(name="read 1777 tokens f32, dim 64", kind="read", tokens=1777, heads=3, dim=64, page=40, dtype="f32",
             padded=5),
        # One user, a short conversation: latency.
        dict(name="single, 1 x 700", kind="single", seqs=1, context=700, ragged=False, queries=1, heads=8, groups=4,
             dim=128, page=16, dtype="bf16", window=0),
        # An ordinary serving batch, contexts of all lengths up to 8192.
        dict(name="single, 32 x up to 8192", kind="single", seqs=32, context=8192, ragged=True, queries=1, heads=8,
             groups=4, dim=128, page=16, dtype="bf16", window=0),
        # Few users with very long contexts.
        dict(name="single, 4 x 131072", kind="single", seqs=4, context=131072, ragged=False, queries=1, heads=8,
             groups=8, dim=128, page=64, dtype="bf16", window=0),
        # Heads that share nothing, four queries each (speculated tokens), a sliding window, heads of 64.
        dict(name="single, 17 x 4 of 5000, window", kind="single", seqs=17, context=5000, ragged=True, queries=4,
             heads=12, groups=1, dim=64, page=32, dtype="f16", window=2048),
        # One whole prompt.
        dict(name="prompt, 4096 of 4096", kind="prompt", seqs=1, context=4096, ragged=False, queries=4096, heads=8,
             groups=4, dim=128, page=64, dtype="bf16", window=0),
        # Chunks of prompts over cached prefixes, ragged.
        dict(name="prompt, 5 x up to 1023 of 9001", kind="prompt", seqs=5, context=9001, ragged=True, queries=1023,
             heads=8, groups=4, dim=128, page=16, dtype="bf16", window=0),
        # Odd sizes throughout: five query heads to a kv head, heads of 96, in float32.
        dict(name="prompt, 3 x up to 777 f32", kind="prompt", seqs=3, context=777, ragged=True, queries=777,
             heads=3, groups=5, dim=96, page=24, dtype="f32", window=0),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["write", "read", "single", "single", "prompt", "prompt"])
    case = dict(kind=kind, heads=rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), dim=rng.choice([64, 80, 96, 128, 128, 192, 256]),
                page=rng.choice([8, 16, 16, 24, 32, 64, 64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    row = case["heads"] * case["dim"]
    if kind in ("write", "read"):
        most = (16384 if kind == "write" else 65536) * 1024 // row
        if case["dtype"] == "f32":
            most //= 2
        case["tokens"] = _log_uniform(rng, 1, min(most, 65536))
        case["padded"] = rng.choice([0, 0, case["tokens"] // 9])
        if kind == "write":
            case["fused"] = rng.random() < 0.5
        return case
    case["groups"] = rng.choice([1, 2, 3, 4, 5, 8, 16]) if case["heads"] <= 8 else rng.choice([1, 2, 4])
    case["ragged"] = rng.random() < 0.6
    case["window"] = rng.choice([0, 0, 0, 128, 1000, 4096])
    if kind == "single":
        case["seqs"] = _log_uniform(rng, 1, 128)
        case["context"] = _log_uniform(rng, 1, min(131072, 4 * 131072 * 1024 // (row * case["seqs"])))
        case["queries"] = min(rng.choice([1, 1, 1, 1, 2, 3, 5]), case["context"])
        return case
    case["seqs"] = _log_uniform(rng, 1, 8)
    most = 5 * 1023 * 9001 * 32 * 128 // (row * case["groups"] * case["seqs"])  # queries times context of a sequence
    if case["dtype"] == "f32":
        most //= 4
    case["context"] = _log_uniform(rng, 32, min(16384, most // 16))
    case["queries"] = _log_uniform(rng, 16, min(case["context"], most // case["context"], 4096))
    return case


def lengths(case):
    """(context length, query count) of every sequence: part of the case, the same for every seed."""
    out = []
    for i in range(case["seqs"]):
        share = 1.0 - 0.93 * ((i * 0.6180339887) % 1.0) if case["ragged"] else 1.0
        context = max(1, int(case["context"] * share))
        queries = case["queries"] if case["kind"] == "single" or not case["ragged"] else max(1, int(case["queries"] * share))
        out.append((context, min(queries, context)))
    return out


def _pairs(case):
    """(visible query-key pairs, keys that any query sees) summed over the sequences."""
    pairs = keys = 0
    for context, queries in lengths(case):
        w = case["window"] or context
        # query at position p sees min(p + 1, w) keys
        pairs += sum(min(p + 1, w) for p in range(context - queries, context))
        keys += min(context, queries - 1 + w)
    return pairs, keys


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    held = case["dim"] // 2 + case["dim"] // GROUP  # bytes of one head's keys (or values) of one token
    if case["kind"] in ("write", "read"):
        real = case["tokens"] - case["padded"]
        # read: what is held, and the values given out; write: the new values and what is held of them before that
        moved = 2 * case["heads"] * (real * held + case["tokens"] * case["dim"] * size) + 8 * case["tokens"]
        if case["kind"] == "write":
            moved += 2 * case["heads"] * real * (case["dim"] * size + held)
        return {"bytes": moved, "flops": 4 * case["heads"] * real * case["dim"]}
    pairs, keys = _pairs(case)
    rows = sum(q for _, q in lengths(case)) * case["heads"] * case["groups"]
    return {"bytes": 2 * case["heads"] * keys * held + rows * (2 * case["dim"] * size + 4),
            "flops": 4 * case["dim"] * case["heads"] * case["groups"] * pairs}


# ------------------------------------------------------------------ the format, in 32 bits

def _encode(x, g):
    """codes [..., dim/2], scales [..., dim/16] of float32 x [..., dim]."""
    y = x.unflatten(-1, (-1, GROUP))
    six = torch.full((), 6.0, device=x.device)
    factor = 2688.0 * torch.ones((), device=x.device) / g
    wanted = y.abs().amax(-1) / six * factor
    scales = wanted.clamp(max=448.0).to(torch.float8_e4m3fn)
    held = scales.float()
    by = torch.where(held == 0, torch.zeros_like(held), factor / held)
    y = y * by.unsqueeze(-1)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales.view(torch.uint8)


def _decode(codes, scales, g):
    """float32 values [..., dim] of codes [..., dim/2] and scales [..., dim/16]."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat([grid, -grid])
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([grid[byte & 15], grid[byte >> 4]], -1)
    values = pairs.index_select(0, codes.reshape(-1).int()).view(*codes.shape[:-1], -1, GROUP)
    by = scales.view(torch.float8_e4m3fn).float() * (g / torch.full((), 2688.0, device=codes.device))
    return (values * by.unsqueeze(-1)).flatten(-2)


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _heads_of(gen, tokens, heads, dim, dtype, channel):
    """Keys or values: normal, each channel with a size of its own (a few channels of keys are large in real models)."""
    return (torch.randn(tokens, heads, dim, generator=gen, device="cuda") * channel).to(dtype)


def _cache(pages, case):
    """An empty cache: pages hold whatever memory held, here bytes 255 (scales that are no number)."""
    shape = (pages, case["heads"], case["page"])
    return {n + part: torch.full(shape + (case["dim"] // per,), 255, dtype=torch.uint8, device="cuda")
            for n in "kv" for part, per in (("_codes", 2), ("_scales", GROUP))}


def _fill(cache, slots, gen, channels, state, page):
    """Random keys and values written into `slots`, some 2^25 values at a time."""
    heads, dim = cache["k_codes"].shape[1], cache["k_codes"].shape[3] * 2
    for at in slots.split(max(1, (1 << 25) // (heads * dim))):
        for n in "kv":
            x = _heads_of(gen, at.numel(), heads, dim, torch.float32, channels[n])
            codes, scales = _encode(x, state["global_" + n])
            cache[n + "_codes"][at // page, :, at % page] = codes
            cache[n + "_scales"][at // page, :, at % page] = scales


def prepare(case, seed):
    gen = _generator(seed)
    heads, dim, page, dtype = case["heads"], case["dim"], case["page"], TYPES[case["dtype"]]
    channels = {n: 1.0 + 3.0 * (torch.rand(heads, dim, generator=gen, device="cuda") < (0.03 if n == "k" else 0.0))
                for n in "kv"}
    state = {"case": dict(case)}
    # fixed global scales, as from a calibration: near the largest magnitude of keys and of values
    state["global_k"] = 22.0 + torch.rand(1, generator=gen, device="cuda")
    state["global_v"] = 6.0 + torch.rand(1, generator=gen, device="cuda")
    if case["kind"] in ("write", "read"):
        tokens = case["tokens"]
        pages = -(-tokens // page) + 3
        cache = _cache(pages, case)
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(tokens, device="cuda") + 2
        if case["kind"] == "write" and tokens <= 256:  # single tokens of as many sequences: each its own page if there are enough
            slots = torch.randperm(pages * page, generator=gen, device="cuda")[:tokens]
        else:
            slots = order[at // page] * page + at % page
        if case["kind"] == "read":
            _fill(cache, slots, gen, channels, state, page)
        if case["padded"]:
            slots[torch.randperm(tokens, generator=gen, device="cuda")[:case["padded"]]] = -1
        state["slots"], state["cache"] = slots, cache
        if case["kind"] == "write":
            if case["fused"]:  # [tokens, 6 heads of them for queries and the rest for keys and values]
                both = torch.empty(tokens, 6 * heads, dim, dtype=dtype, device="cuda")
                both[:, 4 * heads:5 * heads] = _heads_of(gen, tokens, heads, dim, dtype, channels["k"])
                both[:, 5 * heads:] = _heads_of(gen, tokens, heads, dim, dtype, channels["v"])
                state["k"], state["v"] = both[:, 4 * heads:5 * heads], both[:, 5 * heads:]
            else:
                state["k"] = _heads_of(gen, tokens, heads, dim, dtype, channels["k"])
                state["v"] = _heads_of(gen, tokens, heads, dim, dtype, channels["v"])
        return state
    lens = lengths(case)
    need = [-(-c // page) for c, _ in lens]
    pages = sum(need) + 2
    cache = _cache(pages, case)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    begin = 0
    for b, ((context, _), n) in enumerate(zip(lens, need)):
        table[b, :n] = order[begin:begin + n]
        begin += n
        at = torch.arange(context, device="cuda")
        _fill(cache, table[b].long()[at // page] * page + at % page, gen, channels, state, page)
    total = sum(q for _, q in lens)
    starts = [0]
    for _, q in lens:
        starts.append(starts[-1] + q)
    state |= {"cache": cache, "table": table,
              "context": torch.tensor([c for c, _ in lens], dtype=torch.int32, device="cuda"),
              "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
              "max_queries": max(q for _, q in lens), "max_context": max(c for c, _ in lens), "total": total,
              "scale": 1.0 / math.sqrt(dim),
              "q": (torch.randn(total, heads * case["groups"], dim, generator=gen, device="cuda") * 1.5).to(dtype)}
    return state


# ------------------------------------------------------------------ one pass

def _read_plain(s, dtype):
    slots = s["slots"]
    there = (slots >= 0).view(-1, 1, 1)
    at = slots.clamp(min=0)
    page = s["case"]["page"]
    out = {n: _decode(s["cache"][n + "_codes"][at // page, :, at % page], s["cache"][n + "_scales"][at // page, :, at % page],
                      s["global_" + n]) for n in "kv"}
    return {n: torch.where(there, x, torch.zeros_like(x)).to(dtype) for n, x in out.items()}


def _write_plain(s):
    page, cache = s["case"]["page"], s["cache"]
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    k_codes, k_scales = _encode(s["k"][keep].float(), s["global_k"])
    v_codes, v_scales = _encode(s["v"][keep].float(), s["global_v"])
    cache["k_codes"][at // page, :, at % page] = k_codes
    cache["k_scales"][at // page, :, at % page] = k_scales
    cache["v_codes"][at // page, :, at % page] = v_codes
    cache["v_scales"][at // page, :, at % page] = v_scales


def _attention_plain(s):
    case, cache, q = s["case"], s["cache"], s["q"].float()
    page, heads, groups, dim = case["page"], case["heads"], case["groups"], case["dim"]
    seqs = s["table"].shape[0]
    key = torch.arange(s["max_context"], device="cuda")
    at = s["table"][:, key // page].clamp(min=0).long()  # [seqs, keys]
    off = (key % page).expand_as(at)
    real = (key < s["context"].view(-1, 1)).view(seqs, 1, -1, 1)
    k = _decode(cache["k_codes"][at, :, off], cache["k_scales"][at, :, off], s["global_k"]).transpose(1, 2)
    v = _decode(cache["v_codes"][at, :, off], cache["v_scales"][at, :, off], s["global_v"]).transpose(1, 2)
    k = torch.where(real, k, torch.zeros_like(k))  # [seqs, heads, keys, dim]
    v = torch.where(real, v, torch.zeros_like(v))
    # queries padded to [seqs, most, ...]
    n = s["starts"].diff()
    i = torch.arange(s["max_queries"], device="cuda")
    row = (s["starts"][:-1].view(-1, 1) + i).clamp(max=s["total"] - 1).long()
    x = q[row].view(seqs, -1, heads, groups, dim).permute(0, 2, 1, 3, 4).reshape(seqs, heads, -1, dim)
    scores = torch.matmul(x * s["scale"], k.transpose(-1, -2))  # [seqs, heads, most * groups, keys]
    p = (s["context"] - n).view(-1, 1) + i  # position of each query
    sees = key <= p.unsqueeze(-1)
    if case["window"]:
        sees = sees & (key > p.unsqueeze(-1) - case["window"])
    sees = sees.repeat_interleave(groups, 1).unsqueeze(1)
    scores = scores.masked_fill_(~sees, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).squeeze(-1)

    def back(y):  # [seqs, heads, most * groups, ...] -> the real rows
        y = y.unflatten(2, (-1, groups)).transpose(1, 2).flatten(2, 3)
        return y[i < n.view(-1, 1)]

    return {"out": back(out).to(s["q"].dtype), "lse": back(lse)}


def run(s):
    case = s["case"]
    dtype = TYPES[case["dtype"]]
    if not own:
        if case["kind"] == "write":
            _write_plain(s)
        return _read_plain(s, dtype) if case["kind"] in ("write", "read") else _attention_plain(s)
    import nvfp4_block_scaled_amd as nv
    cache = nv.KVCache(**s["cache"], global_scale_k=s["global_k"], global_scale_v=s["global_v"])
    if case["kind"] == "write":
        nv.nvfp4_kv_write(cache, s["k"], s["v"], s["slots"])
    if case["kind"] in ("write", "read"):
        k, v = nv.nvfp4_kv_read(cache, s["slots"], dtype=dtype)
        return {"k": k, "v": v}
    out, lse = nv.nvfp4_kv_attention(s["q"], cache, s["table"], s["context"], query_starts=s["starts"],
                                     max_queries=s["max_queries"], max_context=s["max_context"], scale=s["scale"],
                                     causal=True, window=case["window"], return_lse=True)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ from the definition, in 64 bits

def _levels():
    """The magnitudes of e2m1 and of e4m3 (finite), from their fields."""
    e2m1 = [(m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)) for e in range(4) for m in range(2)]
    e4m3 = [(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127]
    return [torch.tensor(t, dtype=torch.float64, device="cuda") for t in (e2m1, e4m3)]


def _nearest(x, levels):
    """Index of the level nearest to x >= 0; halfway goes to the even index, above the last to the last."""
    up = torch.searchsorted(levels, x.contiguous()).clamp(1, len(levels) - 1)
    low, high = levels[up - 1], levels[up]
    to_up = (x - low > high - x) | ((x - low == high - x) & (up % 2 == 0))
    return torch.where(to_up, up, up - 1)


def _exact_values(x, g):
    """What NVFP4 keeps of x [..., dim], as float64."""
    e2m1, e4m3 = _levels()
    y = x.double().unflatten(-1, (-1, GROUP))
    scale = e4m3[_nearest(y.abs().amax(-1) / 6 * (2688 / g.double()), e4m3)].unsqueeze(-1)
    by = torch.where(scale > 0, 2688 / g.double() / scale.clamp(min=2.0 ** -9), torch.zeros_like(scale))
    kept = e2m1[_nearest((y * by).abs(), e2m1)] * torch.sign(y)
    return (kept * scale * (g.double() / 2688)).flatten(-2)


def _exact_held(codes, scales, g):
    """float64 values of held codes and scales."""
    e2m1, e4m3 = _levels()
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    sign = 1.0 - 2.0 * (both >> 3).double()
    by = torch.cat([e4m3, e4m3.new_tensor([float("nan")])])[(scales & 127).long()]
    return sign * e2m1[both & 7] * by.repeat_interleave(GROUP, -1) * (g.double() / 2688)


def exact(case, seed):
    s = prepare(case, seed)
    page, cache = case["page"], s["cache"]
    if case["kind"] in ("write", "read"):
        at = s["slots"].clamp(min=0)
        out = {}
        for n in "kv":
            if case["kind"] == "write":
                x = torch.cat([_exact_values(t, s["global_" + n]) for t in s[n].split(2048)])
            else:
                x = torch.cat([_exact_held(cache[n + "_codes"][t // page, :, t % page],
                                           cache[n + "_scales"][t // page, :, t % page], s["global_" + n])
                               for t in at.split(8192)])
            x[s["slots"] < 0] = 0.0
            out[n] = x
        return out
    heads, groups, dim = case["heads"], case["groups"], case["dim"]
    out = torch.zeros(s["total"], heads * groups, dim, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], heads * groups, dtype=torch.float64, device="cuda")
    first = 0
    for b, (context, queries) in enumerate(lengths(case)):
        j = torch.arange(context, device="cuda")
        pages, off = s["table"][b].long()[j // page], j % page
        pos = torch.arange(context - queries, context, device="cuda")
        hidden = j > pos.view(-1, 1)
        if case["window"]:
            hidden |= j <= pos.view(-1, 1) - case["window"]
        for h in range(heads):
            k = _exact_held(cache["k_codes"][pages, h, off], cache["k_scales"][pages, h, off], s["global_k"])
            v = _exact_held(cache["v_codes"][pages, h, off], cache["v_scales"][pages, h, off], s["global_v"])
            for at in range(h * groups, (h + 1) * groups):
                logits = s["q"][first:first + queries, at].double() @ k.t() * s["scale"]
                logits.masked_fill_(hidden, float("-inf"))
                lse[first:first + queries, at] = torch.logsumexp(logits, -1)
                out[first:first + queries, at] = torch.softmax(logits, -1) @ v
        first += queries
    return {"out": out, "lse": lse}
