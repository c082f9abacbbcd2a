"""Attention over the NVFP4 cache where the size of the scores, of their factor
or of what a mask hides could spoil a result.  The bound is that of _kv.py."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import _kv
from _parity import say
from test_gpu_kv_attention import _batch, _run

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
MASKS = [(True, 0), (True, 37), (False, 0)]  # causal, window
ROWS = [1, 17]  # queries: few rows a kv head, and many


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    nv.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("queries", ROWS)
@pytest.mark.parametrize("causal,window", MASKS)
def test_zero_global_scales(dtype, dim, queries, causal, window):
    """A global scale of 0 (the largest magnitude of keys or values that are all 0): every score is 0 and the
    output the mean of what is seen, or every output is 0."""
    say(f"global scale 0 {dtype} d{dim} queries {queries} causal {causal} window {window}")
    contexts, counts = [130, 64, queries, 0], [queries, queries, queries, queries]
    for g in ((0.0, 6.0), (20.0, 0.0), (0.0, 0.0)):
        _run(contexts, counts, 1, 2, dim, 16, dtype, 2000 + dim + queries, causal=causal, window=window, g=g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("queries", ROWS)
@pytest.mark.parametrize("causal,window", MASKS)
def test_tiny_queries(dtype, dim, queries, causal, window):
    """Queries around and below the smallest normal number, the scale as usual: the scores are as good as 0."""
    say(f"tiny queries {dtype} d{dim} queries {queries} causal {causal} window {window}")
    contexts, counts = [130, 64, queries, 0], [queries, queries, queries, queries]
    for size, g_k in ((2.0 ** -124, 4.0), (2.0 ** -130, 20.0), (2.0 ** -134, 6.0), (2.0 ** -140, 22.0)):
        _run(contexts, counts, 1, 2, dim, 16, dtype, 2100 + dim + queries, causal=causal, window=window, g=(g_k, 6.0),
             q_size=size)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", ROWS)
def test_other_global_scales(dtype, queries):
    """Negative global scales are factors like others; one that is NaN makes NaN of every query that sees a key,
    and of no other."""
    say(f"global scales below 0 and NaN {dtype} queries {queries}")
    contexts, counts = [130, 64, max(queries - 5, 0), 0], [queries] * 4
    for causal, window in MASKS:
        _run(contexts, counts, 1, 2, 64, 16, dtype, 2300, causal=causal, window=window, g=(-20.0, -6.0))
    table, pages, _ = _batch(contexts, 16, 5)
    cache = _kv.random_cache(pages, 16, 1, 64, 2301, float("nan"), 6.0)
    q = torch.randn(4 * queries, 2, 64, generator=torch.Generator().manual_seed(2302)).to(dtype).cuda()
    starts = torch.arange(5, dtype=torch.int32, device="cuda") * queries
    got, lse = nv.nvfp4_kv_attention(q, cache, table.cuda(), torch.tensor(contexts, dtype=torch.int32, device="cuda"),
                                     query_starts=starts, max_queries=queries, return_lse=True)
    sees = torch.cat([torch.arange(c - queries, c) >= 0 for c in contexts]).cuda()
    assert torch.isnan(got[sees]).all() and torch.isnan(lse[sees]).all()
    assert not got[~sees].any() and (lse[~sees] == float("-inf")).all() and not sees.all()


def _attend(cache, table, contexts, counts, q, scale, causal, window):
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    lens = torch.tensor(contexts, dtype=torch.int32, device="cuda")
    got, lse = nv.nvfp4_kv_attention(q, cache, table.cuda(), lens, scale=scale, causal=causal, window=window,
                                     query_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                                     max_queries=max(counts), max_context=max(contexts), return_lse=True)
    torch.cuda.synchronize()
    return got, lse, starts


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", ROWS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sign", [0, -1])
def test_large_scores(dtype, queries, dim, sign):
    """Scores of 2^16 and far more, of both signs or all negative.  A score's error e (as in _kv.py) is then
    above 1, so that keys whose scores lie within 2 e of the largest may share the output in any way: it lies
    between the least and the greatest of their values, up to the roundings of weights and output.  Keys 40
    below those weigh nothing.  Mostly one key is left, and the output is its value."""
    contexts, counts, page, groups, inf = [600, 130, queries], [queries] * 3, 16, 2, float("inf")
    table, pages, _ = _batch(contexts, page, 5)
    cache = _kv.random_cache(pages, page, 1, dim, 2200 + dim)
    if sign:
        cache.k_codes &= 0x77
    held = {n: getattr(cache, n).cpu()[:, 0] for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    unit = _kv.UNIT[dtype]
    single_float = dtype is torch.float32
    base = torch.randn(sum(counts), groups, dim, generator=torch.Generator().manual_seed(2201 + dim))
    if sign:
        base = -base.abs()
    alone = 0
    for size in (3e4, 1e7, 1e9, 1e30):
        by = min(size, 2e3) if dtype is torch.float16 else size  # (beyond float16: the scale makes up for it)
        q = (base * by).to(dtype)
        scale = dim ** -0.5 * (size / by)
        for causal, window in MASKS:
            what = (dtype, dim, sign, size, causal, window)
            got, lse, starts = _attend(cache, table, contexts, counts, q.cuda(), scale, causal, window)
            assert torch.isfinite(got).all() and torch.isfinite(lse).all(), what
            for b, context in enumerate(contexts):
                j = torch.arange(context)
                at, off = table[b].long()[j // page], j % page
                k = _kv.values(held["k_codes"][at, off], held["k_scales"][at, off], 20.0)
                v = _kv.values(held["v_codes"][at, off], held["v_scales"][at, off], 6.0)
                x = q[starts[b]:starts[b + 1]].double()  # [queries, groups, dim]
                pos = torch.arange(context - queries, context).view(-1, 1, 1)
                hidden = (j > pos) if causal else torch.zeros(queries, 1, context, dtype=torch.bool)
                if window:
                    hidden = hidden | (j <= pos - window)
                s = (x @ k.t() * scale).masked_fill(hidden, -inf)
                most = (x.abs() @ k.abs().t() * scale).masked_fill(hidden, 0.0).amax(-1)
                e = ((dim + 8) * 2.0 ** -24 + (2.0 ** -22 if single_float else 0.0)) * most
                want = torch.logsumexp(s, -1)
                here = slice(starts[b], starts[b + 1])
                assert ((lse[here].cpu().double() - want).abs() <=
                        e + 2.0 ** -20 + context * 2.0 ** -24 + 2.0 ** -22 * want.abs()).all(), what
                near = (s >= (s.amax(-1) - 2 * e - 40).unsqueeze(-1)).unsqueeze(-1)  # [queries, groups, keys, 1]
                alone += int((near.sum(2) == 1).sum())
                low = torch.where(near, v, torch.full_like(v, inf)).amin(2)
                high = torch.where(near, v, torch.full_like(v, -inf)).amax(2)
                slack = ((2.0 ** -22 if single_float else 2.0 ** -11) + unit + 2.0 ** -18) * (1 + 2 * unit) * \
                    torch.maximum(low.abs(), high.abs()) + 1e-12
                o = got[here].cpu().double()
                assert ((o >= low - slack) & (o <= high + slack)).all(), what
    say(f"large scores {dtype} d{dim} queries {queries} sign {sign}: {alone} rows of one key")
    assert alone > 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 31 + 5, 2 ** 40])
@pytest.mark.parametrize("queries", [4, 45])
def test_huge_windows(dtype, window, queries):
    """Windows that hide nothing, also for queries that stand before the context."""
    say(f"window {window} {dtype} queries {queries}")
    _run([1, 3, 200, 0, 60], [queries] * 5, 1, 2, 64, 16, dtype, 2400, window=window)
    _run([1, 3, 200, 0, 60], [queries] * 5, 1, 2, 64, 16, dtype, 2401, window=window)


@pytest.mark.parametrize("queries", [4, 45])
def test_windows_around_the_longest_context(queries):
    """A window as long as max_context is none; one key less hides the first key from the last query."""
    for window in (198, 199, 200, 201):
        _run([200, 199, 3, 60], [queries] * 4, 1, 2, 64, 16, torch.bfloat16, 2402, window=window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [16, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("queries", [4, 13, 45])
@pytest.mark.parametrize("causal,window", MASKS)
def test_values_not_a_number(dtype, dim, queries, causal, window):
    """A held value whose block scale is no number makes NaN of its 16 elements for the queries that see its key,
    and changes no bit of anything else: hidden keys, ends of tiles, a page that is not there beside it, split
    contexts."""
    say(f"values that are no number {dtype} d{dim} queries {queries} causal {causal} window {window}")
    contexts, counts, page, groups = [130, 64, 3000, queries], [queries] * 4, 16, 2
    table, pages, _ = _batch(contexts, page, 7)
    table[0, 6] = -1
    cache = _kv.random_cache(pages, page, 1, dim, 2500 + dim)
    q = torch.randn(sum(counts), groups, dim, generator=torch.Generator().manual_seed(2501)).to(dtype).cuda()
    want, want_lse, starts = _attend(cache, table, contexts, counts, q, dim ** -0.5, causal, window)
    places = [(0, 129, 0), (0, 127, dim // 16 - 1), (0, 95, 0), (0, 112, 0), (1, 63, 0), (1, 62, dim // 32),
              (1, 64 - queries, 0), (2, 2999, dim // 16 - 1), (2, 2960, 0), (2, 5, 0), (3, queries - 1, 0), (3, 1, 0)]
    for b, j, group in places:
        cache.v_scales[int(table[b, j // page]), 0, j % page, group] = 0x7F if j % 2 else 0xFF
        for i in range(queries):
            pos = contexts[b] - queries + i
            if not causal or (j <= pos and (not window or j > pos - window)):
                want[starts[b] + i, :, 16 * group:16 * group + 16] = float("nan")
    got, lse, _ = _attend(cache, table, contexts, counts, q, dim ** -0.5, causal, window)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0)) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [4, 13, 45])
@pytest.mark.parametrize("window", [0, 37])
def test_keys_not_a_number(dtype, queries, window):
    """A held key that is no number makes NaN of the queries that see it; the others keep within their bound."""
    contexts, counts, page, dim = [130, 64, queries], [queries] * 3, 16, 128
    table, pages, _ = _batch(contexts, page, 7)
    cache = _kv.random_cache(pages, page, 1, dim, 2600)
    q = torch.randn(sum(counts), 2, dim, generator=torch.Generator().manual_seed(2601)).to(dtype).cuda()
    lens, starts = torch.tensor(contexts, dtype=torch.int32), [0, queries, 2 * queries, 3 * queries]
    out, ref_lse, bound, lse_bound = _kv.reference(q, cache, table, lens, starts, dim ** -0.5, True, window)
    for b, j in ((0, 128), (1, 63), (2, queries - 2)):
        cache.k_scales[int(table[b, j // page]), 0, j % page, 3] = 0x7F
    got, lse, _ = _attend(cache, table, contexts, counts, q, dim ** -0.5, True, window)
    bad = torch.zeros(3 * queries, dtype=torch.bool)
    for b, j in ((0, 128), (1, 63), (2, queries - 2)):
        pos = torch.arange(contexts[b] - queries, contexts[b])
        bad[starts[b]:starts[b + 1]] = (j <= pos) & (j > pos - window if window else True)
    assert torch.isnan(got[bad.cuda()]).all() and torch.isnan(lse[bad.cuda()]).all() and 0 < bad.sum() < 3 * queries
    off, off_lse = (got.cpu().double() - out).abs(), (lse.cpu().double() - ref_lse).abs()
    assert (off[~bad] <= bound[~bad]).all() and (off_lse[~bad] <= lse_bound[~bad]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [16, 64, 128, 192, 256])
@pytest.mark.parametrize("queries", [1, 13, 45])
@pytest.mark.parametrize("size", [3.0, 8.0, 14.0])
def test_small_weights(dtype, dim, queries, size):
    """Each output element takes its value from keys of one score alone, down to 84 below the largest (a weight of
    2^-121): its own bits are kept, whatever the largest weight."""
    say(f"small weights {dtype} d{dim} queries {queries} size {size}")
    contexts, page = [200, 77], 16
    table, pages, _ = _batch(contexts, page, 9)
    cache = _kv.random_cache(pages, page, 1, dim, 2700, None, None)
    level = torch.arange(page) % 8  # the code, and the element that its keys' values have
    k = torch.zeros(pages, 1, page, dim // 2, dtype=torch.uint8)
    k[:, 0, :, 0] = level.to(torch.uint8)
    v = torch.zeros(pages, 1, page, dim, dtype=torch.uint8)
    v[:, 0, torch.arange(page), level] = torch.randint(1, 8, (pages, page), generator=torch.Generator().manual_seed(2701),
                                                       dtype=torch.uint8)
    cache.k_codes.copy_(k)
    cache.v_codes.copy_(v[..., 0::2] | v[..., 1::2] << 4)
    cache.k_scales.fill_(0x38)
    cache.v_scales.fill_(0x38)
    q = torch.zeros(2 * queries, 2, dim)
    q[:, 0, 0], q[:, 1, 0] = -size, size  # the first heads prefer keys of 0, the second those of 6
    q = q.to(dtype).cuda()
    got, lse, starts = _attend(cache, table, contexts, [queries] * 2, q, 1.0, True, 0)
    lens = torch.tensor(contexts, dtype=torch.int32)
    _kv.check(got, lse, _kv.reference(q, cache, table, lens, starts, 1.0), f"{dtype} d{dim} size {size}")


def test_scales_and_codes_assigned_anew():
    """A cache whose global scales and codes are assigned anew gives what a cache made of them gives."""
    table, pages, _ = _batch([100], 16, 3)
    a, b = (_kv.random_cache(pages, 16, 2, 64, seed, *g) for seed, g in ((1, (20.0, 6.0)), (2, (5.0, 30.0))))
    slots = torch.arange(pages * 16, device="cuda")
    q = torch.randn(1, 4, 64, device="cuda").bfloat16()
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")

    def results(c):
        return [*nv.nvfp4_kv_read(c, slots, dtype=torch.float32), nv.nvfp4_kv_attention(q, c, table.cuda(), lens)]

    old = results(a)
    for n in ("global_scale_k", "global_scale_v", "k_codes", "k_scales", "v_codes", "v_scales"):
        setattr(a, n, getattr(b, n))
    new = results(a)
    assert all(torch.equal(x, y) for x, y in zip(new, results(b)))
    assert not any(torch.equal(x, y) for x, y in zip(new, old))


@pytest.mark.parametrize("counts", [[3, 1, 0, 2], [50, 7, 1, 0], [1, 1, 1, 1]])
def test_query_counts_that_are_not_stated(counts):
    """Without max_queries every query of query_starts is answered, whatever the output's memory held."""
    contexts = [130, 64, 20, 5]
    table, pages, _ = _batch(contexts, 16, 7)
    cache = _kv.random_cache(pages, 16, 2, 64, 2800)
    starts = [sum(counts[:i]) for i in range(5)]
    q = torch.randn(starts[-1], 4, 64, generator=torch.Generator().manual_seed(2801)).bfloat16().cuda()
    lens = torch.tensor(contexts, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"))
    got, lse = nv.nvfp4_kv_attention(q, cache, table.cuda(), lens, return_lse=True, out=out,
                                     query_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    _kv.check(got, lse, _kv.reference(q, cache, table, lens, starts, 0.125), f"counts {counts}")
