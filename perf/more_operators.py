"""Measured cases of a decoder layer's other operators: norm, rotation into the cache, a tree of drafted tokens, experts.

Four kinds of case:
  norm    h = x + residual, its root-mean-square norm, encoded in an mx mode (groups of 32, power-of-two scales)
  rotate  queries and keys rotated by their positions, keys and values quantised into their slots of an NVFP4 cache
  tree    attention of drafted tokens, which form a tree, over the cached context before them and their own ancestors
  moe     router, the chosen experts' gated products on NVFP4 weights, and their weighted sum, for a few tokens

NVFP4: e2m1 codes (two to a byte, element 2j in the low nibble) and one e4m3 scale per 16 values; a value is
e2m1(code) * e4m3(scale) * g / 2688 with a float32 global scale g.

`own` false: elementary torch operations in 32 bits (sums of squares and router logits in 64: a code, and the choice of
an expert, hang on their last bits).  `own` true: the package's calls on the same inputs.
"""
import math

import torch

own = False

GROUP, MX_GROUP = 16, 32
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One token of a decoding step in front of a quantised projection: latency.
        dict(name="norm 1 x 4096", kind="norm", rows=1, k=4096, dtype="bf16", mode="mxfp8", residual=True, packed=True,
             normed=False),
        # A batch of prompts, quantised straight into the operand layout of the block-scaled product.
        dict(name="norm 8192 x 4096", kind="norm", rows=8192, k=4096, dtype="bf16", mode="mxfp8", residual=True,
             packed=True, normed=False),
        # Odd sizes, 4-bit codes in rows, the normed values themselves wanted too (a router reads them).
        dict(name="norm 517 x 1056 f32, mxfp4", kind="norm", rows=517, k=1056, dtype="f32", mode="mxfp4", residual=False,
             packed=False, normed=True),
        # One decoding step of 64 sequences.
        dict(name="rotate 64 single tokens", kind="rotate", tokens=64, heads=8, groups=4, dim=128, rotary=128, page=16,
             length=32768, dtype="bf16", interleaved=False, padded=0),
        # Prompts, straight out of the fused projection.
        dict(name="rotate 16384 prompt tokens", kind="rotate", tokens=16384, heads=8, groups=4, dim=128, rotary=128,
             page=64, length=32768, dtype="bf16", interleaved=False, padded=0),
        # Part of each head rotated, in neighbouring pairs; odd sizes, some tokens of the batch padding.
        dict(name="rotate 2777 tokens, dim 96", kind="rotate", tokens=2777, heads=5, groups=3, dim=96, rotary=64, page=24,
             length=8192, dtype="f16", interleaved=True, padded=19),
        # One user, a short conversation, a tree of 26 drafted tokens: latency.
        dict(name="tree 1 x 26 of 900", kind="tree", seqs=1, context=900, drafts=26, ragged=False, heads=8, groups=4,
             dim=128, page=16, dtype="bf16", window=0),
        # A serving batch, full trees over contexts of all lengths up to 16384.
        dict(name="tree 16 x 64 of up to 16384", kind="tree", seqs=16, context=16384, drafts=64, ragged=True, heads=8,
             groups=4, dim=128, page=16, dtype="bf16", window=0),
        # Heads of 80 in float32, a sliding window, trees of all sizes.
        dict(name="tree 5 x up to 47 f32, window", kind="tree", seqs=5, context=5000, drafts=47, ragged=True, heads=3,
             groups=2, dim=80, page=24, dtype="f32", window=2000),
        # One token, many small experts: latency and the weights of the eight chosen.
        dict(name="moe 1 token, 8 of 64", kind="moe", tokens=1, experts=64, top_k=8, k=2048, f=1024, dtype="bf16"),
        # A small batch on large experts: nearly all of them are read.
        dict(name="moe 16 tokens, 2 of 8", kind="moe", tokens=16, experts=8, top_k=2, k=4096, f=14336, dtype="bf16"),
        # Odd sizes in float32.
        dict(name="moe 7 tokens, 3 of 11 f32", kind="moe", tokens=7, experts=11, top_k=3, k=1040, f=592, dtype="f32"),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    case = _draw(rng)
    most = max((work(c) for c in listed() if c["kind"] == case["kind"]), key=lambda w: w["bytes"])
    size = {"norm": "rows", "rotate": "tokens", "tree": "context", "moe": "f"}[case["kind"]]
    while any(work(case)[n] > most[n] for n in most):  # no more work than the largest listed case
        case[size] = max(case[size] * 3 // 4, case.get("drafts", 0)) // (GROUP if size == "f" else 1) * (GROUP if size == "f" else 1)
    return case


def _draw(rng):
    kind = rng.choice(["norm", "rotate", "tree", "moe"])
    case = dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if kind == "norm":
        case["k"] = MX_GROUP * _log_uniform(rng, 2, 512)
        case["rows"] = _log_uniform(rng, 1, min(65536, 8192 * 4096 // case["k"]) // (2 if case["dtype"] == "f32" else 1))
        case["mode"] = rng.choice(["mxfp8", "mxfp8", "mxfp4"])
        case["packed"] = case["mode"] == "mxfp8" and rng.random() < 0.6
        case["residual"], case["normed"] = rng.random() < 0.7, rng.random() < 0.4
        return case
    if kind == "moe":
        case["experts"] = _log_uniform(rng, 3, 160)
        case["top_k"] = rng.randint(1, min(8, case["experts"]))
        case["tokens"] = _log_uniform(rng, 1, 32)
        case["k"] = GROUP * _log_uniform(rng, 8, 448)
        most = 8 * 4096 * 14336 // (case["experts"] * case["k"] * (2 if case["dtype"] == "f32" else 1))
        case["f"] = GROUP * _log_uniform(rng, 8, max(9, min(896, most // GROUP)))
        return case
    case |= dict(heads=rng.choice([1, 2, 3, 4, 5, 8]), groups=rng.choice([1, 2, 3, 4, 5, 8]),
                 dim=rng.choice([64, 80, 96, 128, 128, 192, 256]), page=rng.choice([8, 16, 16, 24, 32, 64, 64, 128]))
    if kind == "rotate":
        case["rotary"] = rng.choice([case["dim"], case["dim"], case["dim"] // 32 * 16])
        row = case["heads"] * (case["groups"] + 2) * case["dim"] * (2 if case["dtype"] == "f32" else 1)
        case["tokens"] = _log_uniform(rng, 1, min(16384 * 48 * 128 // row, 65536))
        case["padded"] = rng.choice([0, 0, case["tokens"] // 9])
        case["length"] = rng.choice([4096, 32768, 65536])
        case["interleaved"] = rng.random() < 0.4
        return case
    case["seqs"] = _log_uniform(rng, 1, 32)
    case["drafts"] = _log_uniform(rng, 2, 100)
    cost = case["heads"] * case["groups"] * case["dim"] * case["seqs"] * case["drafts"] * (2 if case["dtype"] == "f32" else 1)
    case["context"] = case["drafts"] + _log_uniform(rng, 1, min(65536, 32 * 128 * 16 * 64 * 8192 // cost))
    case["ragged"] = rng.random() < 0.6
    case["window"] = rng.choice([0, 0, 0, 128, 1000, 4096])
    return case


# ------------------------------------------------------------------ trees: part of the case, the same for every seed

def lengths(case):
    """(context length, drafted tokens) of every sequence; the drafts are the last tokens of the context."""
    out = []
    for i in range(case["seqs"]):
        share = 1.0 - 0.93 * ((i * 0.6180339887) % 1.0) if case["ragged"] else 1.0
        drafts = max(1, int(case["drafts"] * share))
        out.append((drafts + max(0, int((case["context"] - case["drafts"]) * share)), drafts))
    return out


def parents(n, i):
    """Parent of each of n drafted tokens of sequence i (-1: it follows the context): a draft's parent is one of the
    eight or so before it."""
    at = []
    for d in range(n):
        step = 1 + int(8 * ((d * 0.7548776662 + i * 0.5698402910) % 1.0))
        at.append(max(-1, d - step) if d else -1)
    return at


def trees(case):
    """Per sequence: lists of the ancestors' bits (itself among them) and of the depths of its drafts."""
    out = []
    for i, (_, n) in enumerate(lengths(case)):
        bits, depth = [], []
        for d, p in enumerate(parents(n, i)):
            bits.append((1 << d) | (bits[p] if p >= 0 else 0))
            depth.append(depth[p] + 1 if p >= 0 else 0)
        out.append((bits, depth))
    return out


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    size = _size(case)
    if case["kind"] == "norm":
        values = case["rows"] * case["k"]
        code = 1.0 if case["mode"] == "mxfp8" else 0.5
        moved = values * (size * (1 + 2 * case["residual"] + case["normed"]) + code + 1 / MX_GROUP) + case["k"] * size
        return {"bytes": moved, "flops": 5 * values}
    if case["kind"] == "moe":
        t, e, k, f = case["tokens"], case["experts"], case["k"], case["f"]
        read = e * (1 - (1 - case["top_k"] / e) ** t)  # experts that some token goes to, on average
        weights = 3 * k * f * (0.5 + 1 / GROUP)
        return {"bytes": read * weights + (2 * t + e) * k * size + t * case["top_k"] * 8,
                "flops": 2 * t * k * (e + 3 * case["top_k"] * f)}
    heads, dim = case["heads"], case["dim"]
    held = dim // 2 + dim // GROUP  # bytes of one head's keys (or values) of one token
    if case["kind"] == "rotate":
        real = case["tokens"] - case["padded"]
        # queries in and out, keys and values in; then what is held of them, read back as values
        moved = case["tokens"] * heads * dim * size * (2 * case["groups"] + 2) + real * (2 * heads * held + 4 * case["rotary"])
        moved += 2 * heads * (real * held + case["tokens"] * dim * size) + 20 * case["tokens"]
        return {"bytes": moved, "flops": case["tokens"] * heads * (3 * case["rotary"] * (case["groups"] + 1) + 4 * dim)}
    pairs = keys = rows = 0
    for (context, n), (bits, depth) in zip(lengths(case), trees(case)):
        before = context - n
        w = case["window"] or context
        pairs += sum(min(before, max(0, w - 1 - d)) for d in depth) + sum(b.bit_count() for b in bits)
        keys += min(before, w - 1) + n
        rows += n * heads * case["groups"]
    return {"bytes": 2 * heads * keys * held + rows * (2 * dim * size + 4), "flops": 4 * dim * heads * case["groups"] * pairs}


# ------------------------------------------------------------------ the formats, in 32 bits

def _encode(x, g):
    """NVFP4 codes [..., dim/2], scales [..., dim/16] of float32 x [..., dim]."""
    y = x.unflatten(-1, (-1, GROUP))
    six = torch.full((), 6.0, device=x.device)
    factor = 2688.0 * torch.ones((), device=x.device) / g
    wanted = y.abs().amax(-1) / six * factor
    scales = wanted.clamp(max=448.0).to(torch.float8_e4m3fn)
    held = scales.float()
    by = torch.where(held == 0, torch.zeros_like(held), factor / held)
    code = _e2m1_codes(y * by.unsqueeze(-1)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales.view(torch.uint8)


def _e2m1_codes(y):
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code + 8 * torch.signbit(y).to(torch.uint8)


def _e2m1_grid(device):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)
    return torch.cat([grid, -grid])


def _decode(codes, scales, g):
    """float32 values [..., dim] of NVFP4 codes [..., dim/2] and scales [..., dim/16]."""
    grid = _e2m1_grid(codes.device)
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([grid[byte & 15], grid[byte >> 4]], -1)
    values = pairs.index_select(0, codes.reshape(-1).int()).view(*codes.shape[:-1], -1, GROUP)
    by = scales.view(torch.float8_e4m3fn).float() * (g / torch.full((), 2688.0, device=codes.device))
    return (values * by.unsqueeze(-1)).flatten(-2)


def _mx_encode(y, mode):
    """(element values [rows, k] as the codes stand for them, scale bytes [rows, k/32]) of float32 y."""
    z = y.unflatten(-1, (-1, MX_GROUP))
    top = torch.full((), 448.0 if mode == "mxfp8" else 6.0, device=y.device)
    u = (z.abs().amax(-1) / top).view(torch.int32)
    byte = ((u >> 23) + ((u & 0x7FFFFF) != 0)).clamp(max=254)
    byte = torch.where(u <= 0x400000, torch.zeros_like(byte), byte)
    z = (z * torch.exp2(127.0 - byte.float()).unsqueeze(-1))
    if mode == "mxfp8":
        values = z.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    else:
        values = _e2m1_grid(y.device)[_e2m1_codes(z).int()]
    return values.flatten(-2), byte.to(torch.uint8)


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _prepare_norm(case, gen, state):
    rows, k, dtype = case["rows"], case["k"], TYPES[case["dtype"]]
    channel = 1.0 + 20.0 * (torch.rand(k, generator=gen, device="cuda") < 0.005)  # a few channels are large in real models
    state["x"] = _randn(gen, rows, k).to(dtype)
    if case["residual"]:
        state["residual"] = (_randn(gen, rows, k) * channel * 2.0).to(dtype)
    state["weight"] = (1.0 + 0.2 * _randn(gen, k)).to(dtype)


def _empty_cache(pages, case):
    """An empty cache: pages hold whatever memory held, here bytes 255 (scales that are no number)."""
    shape = (pages, case["heads"], case["page"])
    return {n + part: torch.full(shape + (case["dim"] // per,), 255, dtype=torch.uint8, device="cuda")
            for n in "kv" for part, per in (("_codes", 2), ("_scales", GROUP))}


def _key_channels(case, gen):
    return 1.0 + 3.0 * (torch.rand(case["heads"], case["dim"], generator=gen, device="cuda") < 0.03)


def _globals(gen, state):
    """Fixed global scales, as from a calibration: near the largest magnitude of keys and of values."""
    state["global_k"] = 22.0 + torch.rand(1, generator=gen, device="cuda")
    state["global_v"] = 6.0 + torch.rand(1, generator=gen, device="cuda")


def _prepare_rotate(case, gen, state):
    tokens, heads, dim, page, dtype = case["tokens"], case["heads"], case["dim"], case["page"], TYPES[case["dtype"]]
    _globals(gen, state)
    pages = -(-tokens // page) + 3
    order = torch.randperm(pages, generator=gen, device="cuda")
    at = torch.arange(tokens, device="cuda") + 2
    if tokens <= 256:  # single tokens of as many sequences, each anywhere in its own
        slots = torch.randperm(pages * page, generator=gen, device="cuda")[:tokens]
        positions = torch.randint(case["length"], (tokens,), generator=gen, device="cuda")
    else:  # prompts
        slots = order[at // page] * page + at % page
        positions = at * 3 // 2 % case["length"]
    if case["padded"]:
        slots[torch.randperm(tokens, generator=gen, device="cuda")[:case["padded"]]] = -1
    # the fused projection's output: queries, keys, values
    nq = heads * case["groups"]
    both = torch.empty(tokens, nq + 2 * heads, dim, dtype=dtype, device="cuda")
    both[:, :nq] = _randn(gen, tokens, nq, dim).to(dtype)
    both[:, nq:nq + heads] = (_randn(gen, tokens, heads, dim) * _key_channels(case, gen)).to(dtype)
    both[:, nq + heads:] = _randn(gen, tokens, heads, dim).to(dtype)
    angle = torch.arange(case["length"], dtype=torch.float64, device="cuda").view(-1, 1) * 10000.0 ** (
        -torch.arange(0, case["rotary"], 2, dtype=torch.float64, device="cuda") / case["rotary"])
    state |= {"q": both[:, :nq], "k": both[:, nq:nq + heads], "v": both[:, nq + heads:], "slots": slots,
              "positions": positions.to(torch.int32), "cache": _empty_cache(pages, case),
              "table": torch.cat([angle.cos(), angle.sin()], -1).float()}  # [length, rotary]: cosines, sines


def _prepare_tree(case, gen, state):
    heads, dim, page, dtype = case["heads"], case["dim"], case["page"], TYPES[case["dtype"]]
    _globals(gen, state)
    channels = {"k": _key_channels(case, gen), "v": torch.ones((), device="cuda")}
    lens = lengths(case)
    need = [-(-c // page) for c, _ in lens]
    pages = sum(need) + 2
    cache = _empty_cache(pages, case)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    begin = 0
    for b, ((context, _), n) in enumerate(zip(lens, need)):
        table[b, :n] = order[begin:begin + n]
        begin += n
        at = torch.arange(context, device="cuda")
        slots = table[b].long()[at // page] * page + at % page
        for some in slots.split(max(1, (1 << 25) // (heads * dim))):
            for n_ in "kv":
                codes, scales = _encode(_randn(gen, some.numel(), heads, dim) * channels[n_], state["global_" + n_])
                cache[n_ + "_codes"][some // page, :, some % page] = codes
                cache[n_ + "_scales"][some // page, :, some % page] = scales
    words = -(-max(n for _, n in lens) // 64)
    tree, positions = [], []
    for (context, n), (bits, depth) in zip(lens, trees(case)):
        for b, d in zip(bits, depth):
            parts = [(b >> (64 * w)) & (2 ** 64 - 1) for w in range(words)]
            tree.append([p - 2 ** 64 if p >= 2 ** 63 else p for p in parts])
            positions.append(context - n + d)
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    state |= {"cache": cache, "table": table, "context": torch.tensor([c for c, _ in lens], dtype=torch.int32, device="cuda"),
              "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"), "total": starts[-1],
              "max_queries": max(n for _, n in lens), "max_context": max(c for c, _ in lens),
              "tree": torch.tensor(tree, dtype=torch.int64, device="cuda"),
              "positions": torch.tensor(positions, dtype=torch.int32, device="cuda"), "scale": 1.0 / math.sqrt(dim),
              "q": (_randn(gen, starts[-1], heads * case["groups"], dim) * 1.5).to(dtype)}


def _prepare_moe(case, gen, state):
    t, e, k, f, dtype = case["tokens"], case["experts"], case["k"], case["f"], TYPES[case["dtype"]]
    state["x"] = _randn(gen, t, k).to(dtype)
    state["router"] = (_randn(gen, e, k) * k ** -0.5).to(dtype)
    for name, n, inner in (("gate_up", 2 * f, k), ("down", k, f)):
        codes = torch.empty(e, n, inner // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(e, n, inner // GROUP, dtype=torch.uint8, device="cuda")
        g = torch.empty(e, device="cuda")
        for i in range(e):
            w = _randn(gen, n, inner) * inner ** -0.5
            g[i] = w.abs().amax()
            codes[i], scales[i] = _encode(w, g[i])
        state |= {name + "_codes": codes, name + "_scales": scales, name + "_global": g}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": dict(case)}
    {"norm": _prepare_norm, "rotate": _prepare_rotate, "tree": _prepare_tree, "moe": _prepare_moe}[case["kind"]](case, gen, state)
    return state


# ------------------------------------------------------------------ one pass, plain

def _operand(case, codes, scales):
    """Codes [rows, k] and scales [rows, k/32]; for the operand of the block-scaled product padded with zeros (scale bytes
    of 0) to tiles of 32 rows and steps of 64 values, the steps to fours: [tiles, 32, steps, 4, 16], [tiles, 32, fours, 4, 2]."""
    if not case["packed"]:
        return {"codes": codes, "scales": scales}
    tiles, quads = -(-case["rows"] // 32), -(-case["k"] // 256)

    def padded(x, columns):
        bits = torch.zeros(32 * tiles, columns, dtype=torch.uint8, device=x.device)
        bits[:x.shape[0], :x.shape[1]] = x.view(torch.uint8)
        return bits.view(x.dtype)

    return {"codes": padded(codes, 256 * quads).view(tiles, 32, 4 * quads, 4, 16),
            "scales": padded(scales, 8 * quads).view(tiles, 32, quads, 4, 2)}


def _norm_plain(s):
    case, x = s["case"], s["x"]
    h = x if not case["residual"] else (x.float() + s["residual"].float()).to(x.dtype)
    mean = h.double().square().mean(-1, keepdim=True)
    r = (1.0 / torch.sqrt(mean + EPS)).float()
    y = h.float() * r * s["weight"].float()
    values, scales = _mx_encode(y, case["mode"])
    out = {"sum": h} if case["residual"] else {}
    if case["normed"]:
        out["normed"] = y.to(x.dtype)
    if case["mode"] == "mxfp8":
        return out | _operand(case, values, scales.view(torch.float8_e8m0fnu))
    by = torch.exp2(scales.float() - 127.0).repeat_interleave(MX_GROUP, -1)
    return out | {"values": (values * by).to(torch.bfloat16)}  # exact: e2m1 times a power of two


def _rotated(x, cos, sin, rotary, interleaved):
    """float32 (or float64) x [tokens, heads, dim] with its first `rotary` values rotated in pairs."""
    if interleaved:
        a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
    else:
        a, b = x[..., :rotary // 2], x[..., rotary // 2:rotary]
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rotary:]], -1)


def _cos_sin(s):
    row = s["table"][s["positions"].long()].unsqueeze(1)
    return row.chunk(2, -1)


def _rotate_plain(s):
    case, cache, page = s["case"], s["cache"], s["case"]["page"]
    cos, sin = _cos_sin(s)
    q = _rotated(s["q"].float(), cos, sin, case["rotary"], case["interleaved"]).to(s["q"].dtype)
    k = _rotated(s["k"].float(), cos, sin, case["rotary"], case["interleaved"])
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    out = {"q": q}
    for n, x in (("k", k[keep]), ("v", s["v"][keep].float())):
        codes, scales = _encode(x, s["global_" + n])
        cache[n + "_codes"][at // page, :, at % page] = codes
        cache[n + "_scales"][at // page, :, at % page] = scales
    at = s["slots"].clamp(min=0)
    for n in "kv":
        x = _decode(cache[n + "_codes"][at // page, :, at % page], cache[n + "_scales"][at // page, :, at % page], s["global_" + n])
        out[n] = torch.where(keep.view(-1, 1, 1), x, torch.zeros_like(x)).to(q.dtype)
    return out


def _tree_plain(s):
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
    n = s["starts"].diff()
    i = torch.arange(s["max_queries"], device="cuda")
    row = (s["starts"][:-1].view(-1, 1) + i).clamp(max=s["total"] - 1).long()  # queries padded to [seqs, most, ...]
    x = q[row].view(seqs, -1, heads, groups, dim).permute(0, 2, 1, 3, 4).reshape(seqs, heads, -1, dim)
    scores = torch.matmul(x * s["scale"], k.transpose(-1, -2))  # [seqs, heads, most * groups, keys]
    before = (s["context"] - n).view(-1, 1, 1)
    p = s["positions"][row].unsqueeze(-1)
    sees = key < before
    if case["window"]:
        sees = sees & (key > p - case["window"])
    draft = (key - before).clamp(min=0)  # [seqs, 1, keys]: which draft a key is
    word = s["tree"][row].gather(-1, (draft // 64).clamp(max=s["tree"].shape[1] - 1).expand(-1, row.shape[1], -1))
    bit = (word >> (draft % 64)) & 1
    sees = sees | ((key >= before) & (key < s["context"].view(-1, 1, 1)) & (bit != 0))
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


def _route(logits, top_k):
    """Indices (ties: the lowest) and softmax weights over the chosen ones, in logits' type."""
    value, index = torch.sort(logits, dim=-1, descending=True, stable=True)
    value, index = value[:, :top_k], index[:, :top_k]
    p = (value - value[:, :1]).exp()
    return index, p / p.sum(-1, keepdim=True)


def _moe_plain(s):
    case, x = s["case"], s["x"]
    index, p = _route(x.double() @ s["router"].double().t(), case["top_k"])
    p = p.float()
    t, pairs = case["tokens"], case["tokens"] * case["top_k"]
    if pairs < case["experts"]:  # the chosen experts' weights, a copy for each pair
        of = index.reshape(-1)
        rows = x.float().repeat_interleave(case["top_k"], 0).unsqueeze(1)
    else:  # every expert for every token
        of = torch.arange(case["experts"], device="cuda")
        rows = x.float()
    weights = _decode(s["gate_up_codes"][of], s["gate_up_scales"][of], s["gate_up_global"][of].view(-1, 1, 1))
    gate, up = torch.matmul(rows, weights.transpose(-1, -2)).chunk(2, -1)  # [pairs, 1, f] or [experts, tokens, f]
    h = gate / (1.0 + torch.exp(-gate)) * up
    weights = _decode(s["down_codes"][of], s["down_scales"][of], s["down_global"][of].view(-1, 1, 1))
    y = torch.matmul(h, weights.transpose(-1, -2))
    if pairs < case["experts"]:
        chosen = y.view(t, case["top_k"], -1)
    else:
        chosen = y[index, torch.arange(t, device="cuda").view(-1, 1)]
    return {"out": (chosen * p.unsqueeze(-1)).sum(1).to(x.dtype), "index": index.to(torch.int32), "weights": p}


# ------------------------------------------------------------------ one pass

def _norm_own(s):
    import nvfp4_block_scaled_amd as nv
    case = s["case"]
    r = nv.nvfp4_mx_rms_norm(s["x"], s["weight"], case["mode"], residual=s.get("residual"), eps=EPS, packed=case["packed"],
                             normed=case["normed"])
    out = {"sum": r.sum} if case["residual"] else {}
    if case["normed"]:
        out["normed"] = r.normed
    rows, k = s["x"].shape
    if case["mode"] != "mxfp8":
        return out | {"values": nv.nvfp4_mx_dequantize(*r.quantized, case["mode"], dtype=torch.bfloat16)}
    if not case["packed"]:
        codes, scales = r.quantized
    else:  # views of the operand as it lies in memory
        tiles, quads = -(-rows // 32), -(-k // 256)
        codes = r.quantized.codes.view(tiles, 4 * quads, 4, 32, 16).permute(0, 3, 1, 2, 4)
        scales = r.quantized.scales.view(tiles, quads, 2, 32, 4).permute(0, 3, 1, 4, 2)
    return out | {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def _cache_own(s):
    import nvfp4_block_scaled_amd as nv
    return nv.KVCache(**s["cache"], global_scale_k=s["global_k"], global_scale_v=s["global_v"])


def _rotate_own(s):
    import nvfp4_block_scaled_amd as nv
    cache = _cache_own(s)
    q = nv.nvfp4_kv_write_rotated(cache, s["k"], s["v"], s["slots"], s["positions"], s["table"], q=s["q"],
                                  interleaved=s["case"]["interleaved"])
    k, v = nv.nvfp4_kv_read(cache, s["slots"], dtype=q.dtype)
    return {"q": q, "k": k, "v": v}


def _tree_own(s):
    import nvfp4_block_scaled_amd as nv
    out, lse = nv.nvfp4_kv_tree_attention(s["q"], _cache_own(s), s["table"], s["context"], s["starts"], s["tree"],
                                          max_queries=s["max_queries"], max_context=s["max_context"], scale=s["scale"],
                                          positions=s["positions"], window=s["case"]["window"], return_lse=True)
    return {"out": out, "lse": lse}


def _moe_own(s):
    import nvfp4_block_scaled_amd as nv
    out, index, weights = nv.nvfp4_moe(s["x"], s["gate_up_codes"], s["gate_up_scales"], s["down_codes"], s["down_scales"],
                                       router=s["router"], top_k=s["case"]["top_k"], global_scale_gate_up=s["gate_up_global"],
                                       global_scale_down=s["down_global"])
    return {"out": out, "index": index, "weights": weights}


def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"norm": _norm_own, "rotate": _rotate_own, "tree": _tree_own, "moe": _moe_own}[kind](s)
    return {"norm": _norm_plain, "rotate": _rotate_plain, "tree": _tree_plain, "moe": _moe_plain}[kind](s)


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
    """What NVFP4 keeps of float64 x [..., dim]."""
    e2m1, e4m3 = _levels()
    y = x.unflatten(-1, (-1, GROUP))
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


def _exact_norm(case, s):
    h = s["x"]
    out = {}
    if case["residual"]:
        h = (h.double() + s["residual"].double()).to(h.dtype)  # the stored sum is what is normed
        out["sum"] = h.double()
    h = h.double()
    y = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / case["k"] + EPS) * s["weight"].double()
    if case["normed"]:
        out["normed"] = y
    e2m1, e4m3 = _levels()
    levels = e4m3 if case["mode"] == "mxfp8" else e2m1
    values, scales = [], []
    for z in y.unflatten(-1, (-1, MX_GROUP)).split(512):
        top = z.abs().amax(-1, keepdim=True) / levels[-1]
        m, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1
        by = torch.ldexp(torch.ones_like(top), torch.where(m == 0.5, e - 1, e).clamp(-127, 127))
        by = torch.where(top == 0, torch.full_like(by, 2.0 ** -127), by)
        kept = levels[_nearest((z / by).abs(), levels)] * torch.sign(z)
        if case["mode"] == "mxfp8":
            values.append(kept.flatten(-2))
            scales.append(by.squeeze(-1))
        else:
            values.append((kept * by).flatten(-2))
    if case["mode"] != "mxfp8":
        return out | {"values": torch.cat(values)}
    codes, scales = torch.cat(values), torch.cat(scales)
    if case["packed"]:
        tiles, quads = -(-case["rows"] // 32), -(-case["k"] // 256)
        more = (0, 256 * quads - codes.shape[1], 0, 32 * tiles - codes.shape[0])
        codes = torch.nn.functional.pad(codes, more).view(tiles, 32, 4 * quads, 4, 16)
        more = (0, 8 * quads - scales.shape[1], 0, 32 * tiles - scales.shape[0])
        scales = torch.nn.functional.pad(scales, more, value=2.0 ** -127).view(tiles, 32, quads, 4, 2)
    return out | {"codes": codes, "scales": scales}


def _exact_rotate(case, s):
    turned = {n: [] for n in "qkv"}
    for part in torch.arange(case["tokens"], device="cuda").split(1024):
        row = s["table"][s["positions"][part].long()].double()
        half = case["rotary"] // 2
        for n in "qkv":
            x = s[n][part].double()
            if n != "v":
                y = x.clone()
                for i in range(half):
                    a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                    c, d = row[:, i:i + 1], row[:, half + i:half + i + 1]
                    y[..., a] = x[..., a] * c - x[..., b] * d
                    y[..., b] = x[..., b] * c + x[..., a] * d
                x = y
            if n != "q":
                x = _exact_values(x, s["global_" + n])
                x[s["slots"][part] < 0] = 0.0
            turned[n].append(x)
    return {n: torch.cat(x) for n, x in turned.items()}


def _exact_tree(case, s):
    page, heads, groups, dim = case["page"], case["heads"], case["groups"], case["dim"]
    out = torch.zeros(s["total"], heads * groups, dim, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], heads * groups, dtype=torch.float64, device="cuda")
    first, cache = 0, s["cache"]
    for b, ((context, n), (bits, depth)) in enumerate(zip(lengths(case), trees(case))):
        j = torch.arange(context, device="cuda")
        pages, off = s["table"][b].long()[j // page], j % page
        hidden = torch.zeros(n, context, dtype=torch.bool, device="cuda")
        if case["window"]:
            hidden |= j <= (context - n + torch.tensor(depth, device="cuda")).view(-1, 1) - case["window"]
        hidden[:, context - n:] = torch.tensor([[not (x >> d) & 1 for d in range(n)] for x in bits], device="cuda")
        for h in range(heads):
            k = _exact_held(cache["k_codes"][pages, h, off], cache["k_scales"][pages, h, off], s["global_k"])
            v = _exact_held(cache["v_codes"][pages, h, off], cache["v_scales"][pages, h, off], s["global_v"])
            for at in range(h * groups, (h + 1) * groups):
                logits = (s["q"][first:first + n, at].double() @ k.t() * s["scale"]).masked_fill_(hidden, float("-inf"))
                lse[first:first + n, at] = torch.logsumexp(logits, -1)
                out[first:first + n, at] = torch.softmax(logits, -1) @ v
        first += n
    return {"out": out, "lse": lse}


def _exact_moe(case, s):
    x, f = s["x"].double(), case["f"]
    logits = torch.stack([(x * row.double()).sum(-1) for row in s["router"]], -1)
    index = torch.argsort(logits, dim=-1, descending=True, stable=True)[:, :case["top_k"]]
    p = torch.softmax(logits.gather(-1, index), -1)
    out = torch.zeros_like(x)
    for e in range(case["experts"]):
        token, place = (index == e).nonzero(as_tuple=True)
        if token.numel() == 0:
            continue
        w = _exact_held(s["gate_up_codes"][e], s["gate_up_scales"][e], s["gate_up_global"][e])
        both = x[token] @ w.t()
        h = both[:, :f] * torch.sigmoid(both[:, :f]) * both[:, f:]
        w = _exact_held(s["down_codes"][e], s["down_scales"][e], s["down_global"][e])
        out.index_add_(0, token, (h @ w.t()) * p[token, place].unsqueeze(-1))
    return {"out": out, "index": index.to(torch.int32), "weights": p}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotate": _exact_rotate, "tree": _exact_tree, "moe": _exact_moe}[case["kind"]](case, s)
